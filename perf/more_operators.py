"""The operators of a beam-search step with per-request adapters, and their plain forms, over the sizes
they are used at.

Three operators meet at the end of such a step: low-rank adapters of many requests are added to a shared
projection (a body's, or the head's logits), each group of beams takes its best continuations over its beams
and the vocabulary (from logits, or from the top-k lists that the fused head returns), and the states that
belong to the beams (token histories, block tables, caches) follow the chosen parents.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run`` makes one pass (the
library's call where ``own`` is true, elementary torch operations where it is false), ``exact`` gives the
result in 64 bits and ``work`` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # draft rows on a draft model's small head, three adapters: launch latency
        dict(name="adapters_tiny", op="adapters", rows=5, H=128, N=4096, R=8, L=3, dtype="bf16", y="f32", ranks=False,
             packed=False, tokens=0),
        # one stream, one token: a square projection of the body with its adapter
        dict(name="adapters_stream", op="adapters", rows=1, H=2560, N=2560, R=16, L=4, dtype="bf16", y="bf16",
             ranks=False, packed=False, tokens=0),
        # a decode batch of eight adapters on the head's fp32 logits, odd rows picked from a packed batch
        dict(name="adapters_head", op="adapters", rows=33, H=2560, N=151936, R=16, L=8, dtype="bf16", y="f32",
             ranks=False, packed=False, tokens=999),
        # many adapters of different ranks at once, hardly two rows share one
        dict(name="adapters_many", op="adapters", rows=64, H=4096, N=128256, R=32, L=48, dtype="f16", y="f16",
             ranks=True, packed=False, tokens=0),
        # packed prompts of eight requests through a body projection
        dict(name="adapters_prompts", op="adapters", rows=16384, H=1024, N=4096, R=64, L=8, dtype="bf16", y="bf16",
             ranks=False, packed=True, tokens=0),
        # four beams of one request over a draft model's vocabulary: launch latency; odd row starts (8200 bytes)
        dict(name="beams_tiny", op="beams", groups=1, beams=4, k=8, V=4100, dtype="f16", mask=False, finished=False,
             keep=False),
        # four beams of one request over fp32 logits; candidates for twice the beams, so that ended ones can leave
        dict(name="beams_single", op="beams", groups=1, beams=4, k=8, V=151936, dtype="f32", mask=False,
             finished=False, keep=False),
        # structured output: few or many tokens are allowed, some beams have ended, survivors keep their slots
        dict(name="beams_grammar", op="beams", groups=16, beams=4, k=4, V=128256, dtype="f32", mask=True,
             finished=True, keep=True),
        # a large batch of wide beams over the largest vocabulary in 16 bits
        dict(name="beams_batch", op="beams", groups=32, beams=8, k=16, V=248320, dtype="bf16", mask=False,
             finished=False, keep=False),
        # beams over the fused head's top-20 lists, no logits in memory
        dict(name="beams_lists", op="lists", groups=64, beams=4, k=8, n=20, V=151936, finished=True, keep=False),
        # token histories, their logprobs and block tables follow the parents into a second set of buffers
        dict(name="reorder_tables", op="reorder", kind="tables", groups=64, beams=4, alive=2, T=2048, in_place=False),
        # the contiguous caches of four layers in place: survivors stay, the other slots are filled from them
        dict(name="reorder_caches", op="reorder", kind="caches", groups=8, beams=4, alive=2, T=2048, layers=4, heads=8,
             D=128, in_place=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; half of them odd."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if rng.random() < 0.5 and n % 2 == 0:
        n = max(lo, n - 1)
    return n


def draw(rng):
    op = rng.choice(["adapters", "adapters", "beams", "beams", "lists", "reorder"])
    if op == "adapters":
        dtype = rng.choice(["bf16", "f16"])
        case = dict(op=op, rows=_spread(rng, 1, 16384), H=8 * _spread(rng, 16, 512), N=_spread(rng, 500, 151936),
                    R=rng.choice([8, 16, 16, 24, 32, 64]), L=_spread(rng, 1, 64), dtype=dtype,
                    y=rng.choice(["f32", dtype]), ranks=rng.random() < 0.5, tokens=0)
        case["packed"] = case["rows"] > 256 or rng.random() < 0.2
        if case["rows"] <= 256 and rng.random() < 0.4:
            case["tokens"] = 999
        case["N"] = min(case["N"], 16384 * 4096 // case["rows"])
        while work(case)["bytes"] > 3e8 or work(case)["flops"] > 1.1e10:
            case["L"], case["N"] = max(1, case["L"] // 2), max(100, case["N"] * 2 // 3)
        return case
    beams = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 16, 32])
    groups = _spread(rng, 1, 256 // beams)
    if op == "reorder":
        kind = rng.choice(["tables", "caches"])
        case = dict(op=op, kind=kind, groups=groups, beams=beams, T=_spread(rng, 16, 2048),
                    in_place=beams > 1 and rng.random() < 0.5)
        case["alive"] = rng.randint(1, beams - 1 if case["in_place"] else beams)
        if kind == "caches":
            case.update(layers=_spread(rng, 1, 8), heads=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 72, 128]))
            while case["T"] > 16 and work(case)["bytes"] > 8e8:
                case["T"] = case["T"] * 2 // 3
        return case
    case = dict(op=op, groups=groups, beams=beams, finished=rng.random() < 0.4)
    case["k"] = rng.choice([1, 2]) * beams
    case["keep"] = case["k"] == beams and rng.random() < 0.5
    if op == "lists":
        case.update(n=rng.choice([5, 8, 20, 32, 64]), V=_spread(rng, 1000, 248320))
        return case
    case.update(V=_spread(rng, 1000, 248320), mask=rng.random() < 0.3)
    case["dtype"] = rng.choice(["bf16", "f16", "f32"]) if groups * beams <= 128 else "bf16"
    return case


def _used(case):
    return min(case["L"], case["rows"])


def _plain_rows(case):
    """Rows without an adapter."""
    return case["rows"] // (case["L"] + 1)


def work(case):
    if case["op"] == "adapters":
        n, H, N = case["rows"], case["H"], case["N"]
        R = (case["R"] + 1) / 2 if case["ranks"] else case["R"]  # (ranks of 1 to R, all as likely)
        some = n - _plain_rows(case)
        return {"bytes": some * H * 2 + _used(case) * R * (H + N) * 2 + 2 * n * N * BYTES[case["y"]],
                "flops": 2 * some * R * (H + N)}
    rows = case["groups"] * case["beams"]
    if case["op"] == "reorder":
        G, B, alive = case["groups"], case["beams"], case["alive"]
        moved, read = (B - alive, min(alive, B - alive)) if case["in_place"] else (B, alive)
        used = sum(_group_lengths(case))
        if case["kind"] == "tables":
            one = used * 8 + G * _pages(case) * 4
        else:
            one = case["layers"] * (used * 2 * case["heads"] * case["D"] * 2 + G * 4096)
        return {"bytes": one * (moved + read) + rows * 8, "flops": 0}
    out = case["groups"] * case["k"] * 12 + rows * 4
    if case["op"] == "lists":
        return {"bytes": rows * case["n"] * 8 + out, "flops": rows * case["n"]}
    V = case["V"]
    return {"bytes": rows * V * BYTES[case["dtype"]] + (rows * ((V + 31) // 32) * 4 if case["mask"] else 0) + out,
            "flops": 4 * rows * V}


def _pages(case):
    return (case["T"] + 15) // 16


def _group_lengths(case):
    """Positions in use, by group: from half of the buffers to all of them."""
    G, T = case["groups"], case["T"]
    return [max(1, T * (G + g + 1) // (2 * G)) for g in range(G)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _adapter_inputs(case, g):
    n, H, N, R, L, dev = case["rows"], case["H"], case["N"], case["R"], case["L"], "cuda"
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    tokens = max(case["tokens"], n)
    s = {"x": randn(tokens, H).to(dt), "a": randn(L, R, H).mul_(H ** -0.5).to(dt), "b": randn(L, N, R).mul_(0.05).to(dt),
         "scales": 0.5 + 1.5 * torch.rand(L, generator=g, device=dev), "ranks": None, "row_idx": None,
         "y": randn(n, N).mul_(2.0).to(DTYPES[case["y"]])}
    # every adapter that fits is in use, and one row in L + 1 has none; packed: a request's rows follow one another
    idx = (torch.arange(n, device=dev) + 1) % (L + 1) - 1
    s["idx"] = (idx.sort().values if case["packed"] else idx[torch.randperm(n, generator=g, device=dev)]).int()
    if case["ranks"]:
        s["ranks"] = torch.randint(1, R + 1, (L,), generator=g, device=dev, dtype=torch.int32)
    if case["tokens"]:
        s["row_idx"] = torch.randint(0, tokens, (n,), generator=g, device=dev, dtype=torch.int32)
    return s


def _beam_scores(case, g):
    rows = case["groups"] * case["beams"]
    s = {"scores": -5.0 - 4.0 * torch.rand(rows, generator=g, device="cuda"), "finished": None}
    if case["finished"]:
        s["finished"] = (torch.rand(rows, generator=g, device="cuda") < 0.15).to(torch.uint8)
    return s


def _beam_inputs(case, g):
    n, V, dev = case["groups"] * case["beams"], case["V"], "cuda"
    # a model's logits: a broad bulk, and a few dozen tokens that stand out, by more in rows the model is sure of
    z = torch.randn(n, V, generator=g, device=dev).mul_(2.0)
    top = torch.randint(0, V, (n, 48), generator=g, device=dev)
    sure = 9.0 + 10.0 * torch.rand(n, 1, generator=g, device=dev)
    z.scatter_reduce_(1, top, sure + 2.0 * torch.randn(n, 48, generator=g, device=dev), "amax")
    s = _beam_scores(case, g)
    s["logits"] = z.to(DTYPES[case["dtype"]])
    s["mask"] = None
    if case["mask"]:
        words = (V + 31) // 32
        share = torch.pow(10.0, -3.0 * torch.rand(n, 1, generator=g, device=dev))
        share = torch.maximum(share, torch.full_like(share, 8.0 / V))
        bits = torch.zeros(n, words * 32, dtype=torch.bool, device=dev)
        bits[:, :V] = torch.rand(n, V, generator=g, device=dev) < share
        bits[:, 0] |= ~bits.any(1)
        place = torch.arange(32, device=dev, dtype=torch.int64)
        packed = (bits.view(n, words, 32).to(torch.int64) << place).sum(-1)
        s["mask"] = (packed - ((packed >> 31) << 32)).to(torch.int32)
    return s


def _list_inputs(case, g):
    n, dev = case["groups"] * case["beams"], "cuda"
    s = _beam_scores(case, g)
    fall = 3.0 * torch.rand(n, case["n"], generator=g, device=dev)
    fall[:, 0] *= 0.5
    s["lp"] = -(fall.cumsum(1) * (0.2 + torch.rand(n, 1, generator=g, device=dev)))
    s["ids"] = torch.rand(n, case["V"], generator=g, device=dev).topk(case["n"], dim=1).indices.int()
    short = torch.rand(n, generator=g, device=dev) < 0.1  # some rows asked for fewer entries
    cut = short[:, None] & (torch.arange(case["n"], device=dev) >= case["n"] // 2)
    s["lp"] = s["lp"].masked_fill(cut, -math.inf)
    s["ids"] = s["ids"].masked_fill(cut, -1)
    return s


def _reorder_inputs(case, g):
    G, B, alive, T, dev = case["groups"], case["beams"], case["alive"], case["T"], "cuda"
    rows = G * B
    # per group `alive` parents; in place they keep their rows and the others take theirs in turn
    order = torch.rand(G, B, generator=g, device=dev).argsort(1)
    turn = torch.arange(B, device=dev) % alive
    if case["in_place"]:
        parents = torch.empty(G, B, dtype=torch.int64, device=dev)
        to = torch.where(torch.arange(B, device=dev) < alive, torch.arange(B, device=dev),
                         (torch.arange(B, device=dev) - alive) % alive)
        parents.scatter_(1, order, order[:, to])
    else:
        parents = order[:, turn].gather(1, torch.rand(G, B, generator=g, device=dev).argsort(1))
    parents = (parents + B * torch.arange(G, device=dev)[:, None]).flatten().int()
    lengths = torch.tensor(_group_lengths(case), dtype=torch.int32, device=dev).repeat_interleave(B)

    def whole(*shape):
        return torch.randint(0, 1 << 30, shape, generator=g, device=dev, dtype=torch.int32)

    if case["kind"] == "tables":  # token history, its logprobs; the block table is moved whole
        tensors = [whole(rows, T), torch.randn(rows, T, generator=g, device=dev), whole(rows, _pages(case))]
        dims, length_dims = [0, 0, 0], [1, 1, None]
    else:  # keys and values of all layers, and a small recurrent state of each layer
        shape = (case["layers"], 2, rows, case["heads"], T, case["D"])
        tensors = [torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16),
                   torch.randn(case["layers"], rows, 1024, generator=g, device=dev)]
        dims, length_dims = [2, 1], [4, None]
    outs = None if case["in_place"] else [torch.zeros_like(t) for t in tensors]
    return {"tensors": tensors, "dims": dims, "length_dims": length_dims, "outs": outs, "parents": parents,
            "lengths": lengths}


INPUTS = {"adapters": _adapter_inputs, "beams": _beam_inputs, "lists": _list_inputs, "reorder": _reorder_inputs}


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return INPUTS[case["op"]](case, g)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        import top_reduction_gb300 as lmh
        state["lmh"] = lmh
        if case["op"] == "adapters":
            state["table"] = lmh.AdapterTable(state["a"], state["b"], scales=state["scales"], ranks=state["ranks"])
        if case["op"] == "reorder":
            state["states"] = lmh.RowStates(state["tensors"], dims=state["dims"], length_dims=state["length_dims"],
                                            outs=state["outs"])
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        lmh = state["lmh"]
        if op == "adapters":
            return lmh.add_adapters(state["x"], state["table"], state["idx"], state["y"], row_idx=state["row_idx"])
        if op == "beams":
            o = lmh.beam_select(state["logits"], state["scores"], case["beams"], k=case["k"],
                                finished=state["finished"], mask=state["mask"], keep_slots=case["keep"])
            return o["scores"], o["parents"], o["tokens"]
        if op == "lists":
            o = lmh.beam_select_lists(state["ids"], state["lp"], state["scores"], case["beams"], k=case["k"],
                                      finished=state["finished"], keep_slots=case["keep"])
            return o["scores"], o["parents"], o["tokens"]
        return lmh.reorder_rows(state["states"], state["parents"], case["beams"], lengths=state["lengths"])
    if op == "adapters":
        return _plain_adapters(state, case)
    if op == "beams":
        z, ids = _plain_best(state, case)
        return _plain_choice(state, case, z, ids)
    if op == "lists":
        lp = state["lp"].double().masked_fill(state["ids"] < 0, -math.inf)
        return _plain_choice(state, case, lp, state["ids"].long())
    return _plain_reorder(state)


def _plain_adapters(s, case):
    """All adapters' products at once; each row keeps its own adapter's."""
    L, R, H, N = case["L"], case["R"], case["H"], case["N"]
    x = s["x"] if s["row_idx"] is None else s["x"][s["row_idx"].long()]
    down = (x.float() @ s["a"].float().view(L * R, H).t()).view(-1, L, R)
    mine = s["idx"][:, None].long() == torch.arange(L, device=x.device)
    down = torch.where(mine[:, :, None], down * s["scales"][:, None], torch.zeros_like(down))
    if s["ranks"] is not None:
        down = torch.where(torch.arange(R, device=x.device) < s["ranks"][:, None], down, torch.zeros_like(down))
    up = s["b"].float().transpose(1, 2).reshape(L * R, N)
    return (s["y"].float() + down.view(-1, L * R) @ up).to(s["y"].dtype)


def _plain_best(s, case):
    """Each row's k best tokens with their logprobs in 64 bits: ties by ascending id, through whole-number keys."""
    z = s["logits"].float() + 0.0  # (-0 becomes +0: they tie)
    V = z.shape[1]
    m = z.amax(1, keepdim=True)
    lse = m.double() + torch.log(torch.exp(z - m).sum(1, keepdim=True, dtype=torch.float64))
    v = torch.arange(V, device=z.device)
    if s["mask"] is not None:
        z = torch.where((s["mask"][:, v // 32] >> (v % 32).int()) & 1 != 0, z, -math.inf)
    bits = z.view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
    best = (order * (1 << 32) + ((1 << 32) - 1 - v)).topk(min(case["k"], V), dim=1).values
    ids = (1 << 32) - 1 - (best & ((1 << 32) - 1))
    return z.gather(1, ids).double() - lse, ids


def _plain_choice(s, case, lp, ids):
    """The best k of each group of beams, from the beams' candidates (best first) and their logprobs."""
    G, B, k = case["groups"], case["beams"], case["k"]
    score = s["scores"].double()[:, None] + lp
    if s["finished"] is not None:  # an ended beam goes on as it is, with the padding token
        done = s["finished"].bool()[:, None]
        first = torch.arange(lp.shape[1], device=lp.device) == 0
        score = torch.where(done, torch.where(first, s["scores"].double()[:, None], -math.inf), score)
        ids = torch.where(done, torch.zeros_like(ids), ids)
    n = score.shape[1]
    best, at = score.view(G, B * n).sort(dim=1, descending=True, stable=True)
    if B * n < k:
        best = torch.nn.functional.pad(best, (0, k - B * n), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, k - B * n))
    best, at = best[:, :k], at[:, :k]
    none = best == -math.inf
    beam = torch.where(none, -1, at // n)
    token = torch.where(none, -1, ids.view(G, B * n).gather(1, at))
    if case["keep"]:
        to = _plain_slots(beam, B)
        best, beam, token = (torch.empty_like(t).scatter_(1, to, t) for t in (best, beam, token))
    base = B * torch.arange(G, device=lp.device)[:, None]
    return best.float(), torch.where(beam < 0, -1, beam + base).int(), token.int()


def _plain_slots(beam, B):
    """Where each candidate goes so that a parent's best child takes the parent's slot, the others the free ones."""
    r = torch.arange(B, device=beam.device)
    again = ((beam[:, :, None] == beam[:, None, :]) & (r[None, :] < r[:, None])).any(2)
    first = ~again & (beam >= 0)
    taken = (first[:, :, None] & (beam[:, :, None] == r)).any(1)
    free = taken.int().sort(dim=1, stable=True).indices
    turn = (~first).long().cumsum(1) - 1
    return torch.where(first, beam, free.gather(1, turn.clamp(min=0)))


def _plain_reorder(s):
    outs = s["outs"] or s["tensors"]
    p = s["parents"].long()
    got = []
    for t, old, dim, along in zip(s["tensors"], outs, s["dims"], s["length_dims"]):
        new = t.index_select(dim, p)
        if along is not None:
            place = [1] * t.dim()
            place[along] = t.shape[along]
            rows = [1] * t.dim()
            rows[dim] = t.shape[dim]
            used = torch.arange(t.shape[along], device=t.device).view(place) < s["lengths"][p].view(rows)
            new = torch.where(used, new, old)
        got.append(new)
    return got


# ---------------------------------------------------------------------------
# the results in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adapters":
        return _exact_adapters(case, s)
    if case["op"] == "reorder":
        return None  # copies: nothing is computed
    return _exact_beams(case, s)


def _exact_adapters(case, s):
    """Adapter by adapter, over the rows that use it."""
    out = s["y"].double()
    rows_of = s["idx"].tolist()
    ranks = None if s["ranks"] is None else s["ranks"].tolist()
    for l in sorted(set(rows_of) - {-1}):
        rows = torch.tensor([i for i, j in enumerate(rows_of) if j == l], device=out.device)
        x = s["x"].index_select(0, rows if s["row_idx"] is None else s["row_idx"].long()[rows]).double()
        r = case["R"] if ranks is None else ranks[l]
        h = torch.einsum("nh,rh->nr", x, s["a"][l, :r].double()) * float(s["scales"][l])
        out[rows] += torch.einsum("nr,vr->nv", h, s["b"][l, :, :r].double())
    return out


def _exact_beams(case, s):
    """Group by group, over all candidates of its beams; the whole numbers come with the scores."""
    G, B, k = case["groups"], case["beams"], case["k"]
    scores, parents, tokens = [], [], []
    cum = s["scores"].tolist()
    ended = [0] * (G * B) if s["finished"] is None else s["finished"].tolist()
    for g in range(G):
        found = []  # (-score, beam, token)
        for b in range(B):
            row = g * B + b
            if ended[row]:
                found.append((-cum[row], b, 0))
                continue
            if case["op"] == "lists":
                lp, ids = s["lp"][row].double(), s["ids"][row].long()
                lp, ids = lp[ids >= 0], ids[ids >= 0]
            else:
                z = s["logits"][row].double()
                lp = z - torch.logsumexp(z, 0)
                ids = torch.arange(case["V"], device=z.device)
                if s["mask"] is not None:
                    place = torch.arange(32, device=z.device, dtype=torch.int32)
                    allowed = ((s["mask"][row][:, None] >> place) & 1).flatten()[:case["V"]].bool()
                    lp, ids = lp[allowed], ids[allowed]
                kth = lp.topk(min(k, lp.numel())).values[-1]
                lp, ids = lp[lp >= kth], ids[lp >= kth]
            found += [(-(cum[row] + v), b, t) for v, t in zip(lp.tolist(), ids.tolist())]
        found = sorted(found)[:k]
        found += [(math.inf, -1, -1)] * (k - len(found))
        if case["keep"]:
            placed = [None] * B
            left = []
            for f in found:
                if f[1] >= 0 and placed[f[1]] is None:
                    placed[f[1]] = f
                else:
                    left.append(f)
            found = [left.pop(0) if f is None else f for f in placed]
        scores.append([-f[0] for f in found])
        parents.append([-1 if f[1] < 0 else g * B + f[1] for f in found])
        tokens.append([f[2] for f in found])
    return (torch.tensor(scores, dtype=torch.float64).cuda(), torch.tensor(parents, dtype=torch.int32).cuda(),
            torch.tensor(tokens, dtype=torch.int32).cuda())
