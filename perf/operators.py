"""The decode-side operators and their plain forms, over the sizes they are used at.

Three operators meet in one decode step around a model body whose embedding and
head share a table held in 4 bits: the table lookup of the last drawn tokens, the
4-bit head projection of the body's rows, and the filtered draw from its logits.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU, ``run``
makes one pass (the library's call where ``own`` is true, elementary torch
operations where it is false), ``exact`` gives the result in 64 bits and ``work``
the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

LOG2E = 1.4426950408889634
FLT_MAX = torch.finfo(torch.float32).max
FRACTION = 2.0 ** 32  # a draw's integer weights have 32 fractional bits
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a handful of draft rows of a small vocabulary: launch latency; odd row starts (8200-byte rows)
        dict(name="sample_tiny", op="sample", rows=5, V=4100, dtype="f16", filters="mixed", mask=False),
        # one chat stream: one row of the fp32 logits a head writes, with the usual top-k and top-p
        dict(name="sample_single", op="sample", rows=1, V=128256, dtype="f32", filters="topk_topp", mask=False),
        # a decode batch of requests with their own settings, greedy and unfiltered ones among them
        dict(name="sample_decode", op="sample", rows=32, V=151936, dtype="f32", filters="mixed", mask=False),
        # structured output: a grammar leaves few or many tokens of each row, min-p on what is left
        dict(name="sample_grammar", op="sample", rows=64, V=128256, dtype="bf16", filters="minp", mask=True),
        # a large decode batch over the largest vocabulary in 16 bits
        dict(name="sample_batch", op="sample", rows=256, V=248320, dtype="bf16", filters="mixed", mask=False),
        # a draft model's small head
        dict(name="q4_tiny", op="project", rows=5, H=128, V=4096, group=32, zeros=False, dtype="bf16", out="f32",
             scales="bf16", tokens=0),
        # one decode stream through a 4-bit head
        dict(name="q4_single", op="project", rows=1, H=2560, V=151936, group=64, zeros=False, dtype="bf16", out="f32",
             scales="bf16", tokens=0),
        # eight sampled rows of packed prompts: rows are picked by index, small groups
        dict(name="q4_prompts", op="project", rows=8, H=1024, V=151936, group=32, zeros=False, dtype="bf16", out="f32",
             scales="f16", tokens=16384),
        # sixteen streams, zero points, 16-bit floats in and out
        dict(name="q4_zeros", op="project", rows=16, H=4096, V=128256, group=128, zeros=True, dtype="f16", out="f16",
             scales="f16", tokens=0),
        # a decode batch
        dict(name="q4_batch", op="project", rows=32, H=2560, V=151936, group=64, zeros=False, dtype="bf16", out="f32",
             scales="bf16", tokens=0),
        # the next step's input rows of a decode batch
        dict(name="lookup_decode", op="lookup", rows=32, H=2560, V=151936, group=64, zeros=False, out="bf16",
             scales="bf16"),
        # the prompt tokens of a prefill
        dict(name="lookup_prompts", op="lookup", rows=16384, H=1024, V=151936, group=32, zeros=True, out="bf16",
             scales="f16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; half of them odd."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if rng.random() < 0.5 and n % 2 == 0:
        n = max(lo, n - 1)
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["sample", "project", "lookup"])
    if op == "sample":
        V = _spread(rng, 1000, 248320)
        rows = _spread(rng, 1, 256)
        return dict(op=op, rows=rows, V=V, dtype=rng.choice(["bf16", "f16", "f32"]) if rows <= 128 else "bf16",
                    filters=rng.choice(["mixed", "mixed", "topk_topp", "minp"]), mask=rng.random() < 0.3)
    group = rng.choice([32, 64, 128])
    H = group * _spread(rng, 1, 4096 // group)
    H = H + group if H == 3072 else H
    V = _spread(rng, 1000, 151936)
    if H * V > 4096 * 128256:
        V = 4096 * 128256 // H
    case = dict(op=op, H=H, V=V, group=group, zeros=rng.random() < 0.5, scales=rng.choice(["bf16", "f16"]))
    if op == "project":
        case.update(rows=_spread(rng, 1, 32), dtype=rng.choice(["bf16", "f16"]), tokens=rng.choice([0, 0, 999]))
        case["out"] = rng.choice(["f32", case["dtype"]])
    else:
        rows = _spread(rng, 1, 16384)
        case.update(rows=min(rows, 16384 * 1024 // H), out=rng.choice(["bf16", "f16", "f32"]))
    return case


def work(case):
    n, V = case["rows"], case["V"]
    if case["op"] == "sample":
        b = n * V * BYTES[case["dtype"]] + (n * ((V + 31) // 32) * 4 if case["mask"] else 0) + n * 28
        return {"bytes": b, "flops": 4 * n * V}
    H, groups = case["H"], case["H"] // case["group"]
    row = H // 2 + groups * (BYTES[case["scales"]] + (1 if case["zeros"] else 0))
    if case["op"] == "project":
        return {"bytes": V * row + n * H * 2 + n * V * BYTES[case["out"]], "flops": 2 * n * V * H}
    return {"bytes": n * (4 + row + H * BYTES[case["out"]]), "flops": 2 * n * H}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sample_inputs(case, g):
    n, V, dev = case["rows"], case["V"], "cuda"
    # a model's logits: a broad bulk, and a few dozen tokens that stand out, by more in rows the model is sure of
    z = torch.randn(n, V, generator=g, device=dev).mul_(2.0)
    top = torch.randint(0, V, (n, 48), generator=g, device=dev)
    sure = 9.0 + 10.0 * torch.rand(n, 1, generator=g, device=dev)
    lift = sure + 2.0 * torch.randn(n, 48, generator=g, device=dev)
    z.scatter_reduce_(1, top, lift, "amax")
    logits = z.to(DTYPES[case["dtype"]])

    def uniform():
        return torch.rand(n, generator=g, device=dev)

    def off(t, value, share):  # some requests leave a filter off
        return torch.where(uniform() < share, torch.full_like(t, value), t)

    s = {"logits": logits, "uniforms": uniform(), "temperature": 0.5 + 0.8 * uniform(),
         "top_k": None, "top_p": None, "min_p": None, "mask": None}
    sizes = torch.tensor([5, 20, 40, 50, 64, 100], dtype=torch.int32, device=dev)
    picks = torch.randint(0, sizes.numel(), (n,), generator=g, device=dev)
    if case["filters"] in ("mixed", "topk_topp"):
        s["top_k"] = sizes[picks]
        s["top_p"] = 0.8 + 0.19 * uniform()
    if case["filters"] in ("mixed", "minp"):
        s["min_p"] = 0.01 + 0.09 * uniform()
    if case["filters"] == "mixed":
        s["temperature"] = off(s["temperature"], 0.0, 0.15)
        s["top_k"] = off(s["top_k"], 0, 0.5)
        s["top_p"] = off(s["top_p"], 1.0, 0.3)
        s["min_p"] = off(s["min_p"], 0.0, 0.7)
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


def _table(case, g):
    """A [V, H] weight of N(0, 0.02) rounded to 4 bits per group, as a loader of a quantised checkpoint has it."""
    V, H, G = case["V"], case["H"], case["group"]
    w = torch.randn(V, H // G, G, generator=g, device="cuda").mul_(0.02)
    dt = DTYPES[case["scales"]]
    zeros = None
    if case["zeros"]:
        lo, hi = w.amin(-1), w.amax(-1)
        scales = ((hi - lo) / 15).to(dt)
        s = scales.float()
        zero = torch.clamp(torch.round(-lo / s), 0, 15)
        q = torch.clamp(torch.round(w / s[..., None]) + zero[..., None], 0, 15)
        zeros = zero.to(torch.uint8)
    else:
        scales = (w.abs().amax(-1) / 7).to(dt)
        q = torch.clamp(torch.round(w / scales.float()[..., None]), -8, 7) + 8
    q = q.to(torch.uint8).view(V, H // 2, 2)
    return {"packed": (q[..., 0] | (q[..., 1] << 4)).contiguous(), "scales": scales.contiguous(), "zeros": zeros}


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    if case["op"] == "sample":
        return _sample_inputs(case, g)
    s = _table(case, g)
    if case["op"] == "project":
        tokens = max(case["tokens"], case["rows"])
        s["hidden"] = torch.randn(tokens, case["H"], generator=g, device="cuda").to(DTYPES[case["dtype"]])
        s["row_idx"] = None
        if case["tokens"]:
            s["row_idx"] = torch.randint(0, tokens, (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
    else:
        s["ids"] = torch.randint(0, case["V"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32)
    return s


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = dict(case)
    if own:
        import top_reduction_gb300 as lmh
        state["lmh"] = lmh
        if case["op"] != "sample":
            state["table"] = lmh.Q4Table(state["packed"], state["scales"], state["zeros"], case["group"])
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        lmh = state["lmh"]
        if case["op"] == "sample":
            o = lmh.sample_from_logits(state["logits"], state["uniforms"], temperature=state["temperature"],
                                       top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"],
                                       mask=state["mask"])
            return o["sampled_ids"], o["sampled_logprob"]
        if case["op"] == "project":
            return lmh.project_q4(state["hidden"], state["table"], row_idx=state["row_idx"],
                                  out_dtype=DTYPES[case["out"]])
        return lmh.lookup_q4(state["ids"], state["table"], scale=math.sqrt(case["H"]), out_dtype=DTYPES[case["out"]])
    if case["op"] == "sample":
        return _plain_sample(state)
    if case["op"] == "project":
        x = state["hidden"] if state["row_idx"] is None else state["hidden"][state["row_idx"].long()]
        w = _plain_weights(state, case, slice(None))
        return (x.float() @ w.t()).to(DTYPES[case["out"]])
    w = _plain_weights(state, case, state["ids"].long())
    return (w * math.sqrt(case["H"])).to(DTYPES[case["out"]])


def _plain_weights(state, case, rows):
    packed = state["packed"][rows]
    n = packed.shape[0]
    q = torch.stack((packed & 15, packed >> 4), -1).float().view(n, -1, case["group"])
    zero = 8.0 if state["zeros"] is None else state["zeros"][rows].float()[..., None]
    return ((q - zero) * state["scales"][rows].float()[..., None]).view(n, case["H"])


def _plain_sample(s):
    z = s["logits"].float()
    n, V = z.shape
    if s["mask"] is not None:
        v = torch.arange(V, device=z.device)
        z = torch.where((s["mask"][:, v // 32] >> (v % 32).to(torch.int32)) & 1 != 0, z, -math.inf)
    zm = z.amax(1, keepdim=True)
    T = s["temperature"][:, None]
    greedy = ~(T > 0)
    c = torch.clamp(torch.reciprocal(torch.where(greedy, torch.ones_like(T), T)) * LOG2E, max=FLT_MAX)
    t = (z - zm) * c
    w = torch.round(torch.exp2(t) * FRACTION).to(torch.int64)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    cum = ws.cumsum(1)
    rank = torch.arange(V, device=z.device)
    keep = torch.ones_like(ws, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"][:, None].long()
        keep &= rank < torch.where((k <= 0) | (k > V), torch.full_like(k, V), k)
    if s["top_p"] is not None:
        p = s["top_p"][:, None]
        mass = (ws * keep).sum(1, keepdim=True)
        need = torch.ceil(p.double() * mass.double()).to(torch.int64).clamp(min=1)
        keep &= (cum - ws < need) | (p >= 1)
    if s["min_p"] is not None:
        m = s["min_p"][:, None]
        keep &= (t.gather(1, order) >= torch.log2(m).clamp(max=0)) | (m <= 0)
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order, ws * keep)
    cdf = kept.cumsum(1)
    total = cdf[:, -1:]
    r = torch.floor(s["uniforms"][:, None].double() * total.double()).to(torch.int64)
    r = torch.minimum(r, total - 1)
    ids = torch.searchsorted(cdf, r, right=True)
    ids = torch.where(greedy, order[:, :1], ids)
    lp = t.gather(1, ids) * math.log(2.0) - torch.log(total.float() / FRACTION)
    lp = torch.where(greedy, torch.zeros_like(lp), lp)
    return ids[:, 0].to(torch.int32), lp[:, 0]


# ---------------------------------------------------------------------------
# the results in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    G = case["group"]
    if case["op"] == "project":
        x = s["hidden"].double()
        if s["row_idx"] is not None:
            x = x.index_select(0, s["row_idx"].long())
        out = torch.empty(case["rows"], case["V"], dtype=torch.float64, device="cuda")
        for v0 in range(0, case["V"], 16384):
            rows = torch.arange(v0, min(v0 + 16384, case["V"]), device="cuda")
            out[:, v0:v0 + rows.numel()] = torch.einsum("nh,vh->nv", x, _exact_rows(s, rows, G))
        return out
    return _exact_rows(s, s["ids"].long(), G) * math.sqrt(case["H"])


def _exact_rows(s, rows, G):
    """Rows of the table in 64 bits."""
    p = s["packed"].index_select(0, rows)
    w = torch.empty(p.shape[0], 2 * p.shape[1], dtype=torch.float64, device=p.device)
    w[:, 0::2] = (p % 16).double()
    w[:, 1::2] = torch.div(p, 16, rounding_mode="floor").double()
    if s["zeros"] is None:
        w -= 8
    else:
        w -= s["zeros"].index_select(0, rows).double().repeat_interleave(G, 1)
    return w * s["scales"].index_select(0, rows).double().repeat_interleave(G, 1)


def _exact_sample(case, s):
    """Row by row. A draw is defined on whole-number weights, the fp32 values 2^t rounded to 32 fractional bits:
    these are taken as they are, all sums are whole numbers, and the log-probability is worked out in 64 bits."""
    n, V = case["rows"], case["V"]
    ids = torch.empty(n, dtype=torch.int32)
    lps = torch.empty(n, dtype=torch.float64)

    def param(name, default):
        return [default] * n if s[name] is None else s[name].tolist()

    T, K, P, M = s["temperature"].tolist(), param("top_k", 0), param("top_p", 1.0), param("min_p", 0.0)
    for i in range(n):
        z = s["logits"][i].double()
        if s["mask"] is not None:
            shifts = torch.arange(32, device=z.device, dtype=torch.int32)
            allowed = ((s["mask"][i][:, None] >> shifts) & 1).flatten()[:V].bool()
            z = z.masked_fill(~allowed, -math.inf)
        best = z.max()
        if not T[i] > 0:
            ids[i], lps[i] = int((z == best).nonzero()[0]), 0.0
            continue
        c32 = min(float((1.0 / s["temperature"][i]).float() * LOG2E), FLT_MAX)
        t32 = (z - best).float() * c32
        weight = (torch.exp2(t32).double() * FRACTION).round().long()
        zs, perm = z.sort(descending=True, stable=True)
        upto = weight[perm].cumsum(0)
        cut = V if K[i] <= 0 else min(int(K[i]), V)
        if P[i] < 1:
            need = max(1, math.ceil(P[i] * int(upto[cut - 1])))
            cut = min(cut, int((upto < need).sum()) + 1)
        if M[i] > 0:
            floor = min(float(torch.log2(s["min_p"][i])), 0.0)
            cut = max(1, min(cut, int((t32 >= floor).sum())))
        chosen = perm[:cut].sort().values
        mass = weight[chosen].cumsum(0)
        total = int(mass[-1])
        u = float(s["uniforms"][i])
        r = min(math.floor(u * total), total - 1)
        j = int(chosen[int((mass <= r).sum())])
        scaled = (z - best) / T[i]
        ids[i] = j
        lps[i] = float(scaled[j] - torch.log(torch.exp(scaled[chosen]).sum()))
    return ids.cuda(), lps.cuda()
