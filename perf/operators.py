"""Cases of the 4-bit codes (encode / decode, scores) and of the sampler.

`run` computes each operator in plain torch operations, or, with `own` set, through the
package's public calls; `exact` gives the same results from the definitions in 64 bits.

  encode   rows -> 4-bit codes with one power-of-two scale per 32 values -> rows again
  scores   alpha * Q X^T + bias, X kept as codes, Q encoded in the call
  sample   one draw per row of logits: temperature, top-k, top-p, min-p, given uniforms
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32                                              # values per scale
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)         # magnitudes of a 4-bit code
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a request's query vectors: short odd rows, the launch latency counts
        {"name": "encode_queries", "op": "encode", "n": 257, "d": 100, "dtype": "f32"},
        # one batch of vectors added to a 128-dimensional index
        {"name": "encode_batch", "op": "encode", "n": 100000, "d": 128, "dtype": "f32"},
        # a whole collection of high-dimensional bf16 embeddings
        {"name": "encode_collection", "op": "encode", "n": 1000000, "d": 960, "dtype": "bf16"},
        # one query against every vector of an index: the codes are read once
        {"name": "scores_one_query", "op": "scores", "m": 1, "n": 1000000, "d": 128,
         "dtype": "f32", "out": "f32", "bias": False},
        # a ragged request batch against high-dimensional vectors, with -|x|^2/2 as the bias (L2 order)
        {"name": "scores_request_batch", "op": "scores", "m": 37, "n": 100003, "d": 960,
         "dtype": "bf16", "out": "f32", "bias": True},
        # a thousand queries of a 128-dimensional index: bound by the scores written
        {"name": "scores_many_queries", "op": "scores", "m": 1000, "n": 100003, "d": 128,
         "dtype": "f32", "out": "f32", "bias": True},
        # a few hidden vectors through an output projection
        {"name": "scores_few_tokens", "op": "scores", "m": 64, "n": 16384, "d": 4096,
         "dtype": "bf16", "out": "bf16", "bias": False},
        # a long prompt's hidden vectors through the same projection: bound by the products
        {"name": "scores_prompt", "op": "scores", "m": 4096, "n": 16384, "d": 4096,
         "dtype": "bf16", "out": "bf16", "bias": False},
        # one answer being written: a single row, latency
        {"name": "sample_one_row", "op": "sample", "rows": 1, "v": 50021, "dtype": "f32",
         "kind": "logits", "topk": True, "topp": True, "minp": False},
        # a serving batch with every request's own settings
        {"name": "sample_batch", "op": "sample", "rows": 64, "v": 50001, "dtype": "bf16",
         "kind": "logits", "topk": True, "topp": True, "minp": True},
        # a draw of a component per point from soft-assignment scores (K = 1024)
        {"name": "sample_components", "op": "sample", "rows": 4096, "v": 1024, "dtype": "f32",
         "kind": "mixture", "topk": False, "topp": False, "minp": True},
        # a large batch over a large vocabulary
        {"name": "sample_large", "op": "sample", "rows": 256, "v": 131072, "dtype": "f32",
         "kind": "logits", "topk": False, "topp": True, "minp": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["encode", "scores", "scores", "sample", "sample"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "encode":
        d = _log_int(rng, 1, 4096)
        n = _log_int(rng, 1, min(1000000, 400000000 // d))
        return {"op": op, "n": n, "d": d, "dtype": dtype}
    if op == "scores":
        d = _log_int(rng, 8, 4096)
        n = _log_int(rng, 100, min(1000000, 67108864 // d))
        m = _log_int(rng, 1, min(4096, max(1, 67108864 // n)))
        return {"op": op, "m": m, "n": n, "d": d, "dtype": dtype,
                "out": rng.choice(["f32", "bf16"]), "bias": rng.random() < 0.5}
    v = _log_int(rng, 2, 262144)
    rows = _log_int(rng, 1, min(4096, max(1, 33554432 // v)))
    return {"op": op, "rows": rows, "v": v, "dtype": dtype,
            "kind": rng.choice(["logits", "logits", "mixture"]), "topk": rng.random() < 0.5,
            "topp": rng.random() < 0.5, "minp": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _vectors(g, n, d, dtype):
    """Embedding-like rows: dimensions of unequal spread and a few outlying values."""
    x = torch.randn(n, d, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(torch.rand(d, generator=g, device="cuda") * 3 - 2)
    far = torch.randint(0, d, (max(1, d // 64),), generator=g, device="cuda")
    x[:, far] *= 8
    return x.to(DTYPES[dtype])


def _scale_tiles(scale_bytes, n, d):
    """Row-major scale bytes [n, blocks] in tiles of 128 rows x 4 blocks (512 bytes): row r,
    block b of a tile at (r % 32) * 16 + (r // 32) * 4 + b."""
    nb = -(-d // BLOCK)
    rt, bt = -(-n // 128), -(-nb // 4)
    full = torch.zeros(rt * 128, bt * 4, dtype=torch.uint8, device=scale_bytes.device)
    full[:n, :nb] = scale_bytes
    return full.view(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "encode":
        return {"case": case, "x": _vectors(g, case["n"], case["d"], case["dtype"])}
    if case["op"] == "scores":
        x = _vectors(g, case["n"], case["d"], "f32")
        codes, scales = _encode_plain(x)
        bias = -0.5 * (x * x).sum(1) if case["bias"] else None
        alpha = 1.0 if case["bias"] else 1.0 / math.sqrt(case["d"])
        return {"case": case, "q": _vectors(g, case["m"], case["d"], case["dtype"]), "codes": codes,
                "scales": _scale_tiles(scales, case["n"], case["d"]), "bias": bias, "alpha": alpha}
    r, v = case["rows"], case["v"]
    if case["kind"] == "logits":       # a model's scores: a broad body and a few likely tokens
        x = torch.randn(r, v, generator=g, device="cuda") * 2.5
        for _ in range(8):
            at = torch.randint(0, v, (r, 1), generator=g, device="cuda")
            x.scatter_(1, at, torch.rand(r, 1, generator=g, device="cuda") * 8 + 6)
    else:                              # log densities of mixture components, far apart
        x = -0.5 * (torch.randn(r, v, generator=g, device="cuda") * 4 + 9) ** 2
    gone = torch.rand(r, 1, generator=g, device="cuda") < 0.3     # rows with forbidden tokens
    x.masked_fill_(gone & (torch.rand(r, v, generator=g, device="cuda") < 0.2), -math.inf)
    state = {"case": case, "logits": x.to(DTYPES[case["dtype"]]),
             "u": torch.rand(r, generator=g, device="cuda", dtype=torch.float64)}
    t = torch.rand(r, generator=g, device="cuda") * 1.2 + 0.3
    t[torch.rand(r, generator=g, device="cuda") < 0.1] = 0.0      # greedy rows
    state["temperature"] = t
    top = min(v, 200)
    k = torch.randint(0, top + 1, (r,), generator=g, device="cuda", dtype=torch.int32)
    state["top_k"] = k if case["topk"] else None
    p = torch.rand(r, generator=g, device="cuda") * 0.5 + 0.5
    state["top_p"] = p if case["topp"] else None
    state["min_p"] = torch.rand(r, generator=g, device="cuda") * 0.1 if case["minp"] else None
    return state


# ------------------------------------------------------------------ plain forms
def _blocks(x):
    n, d = x.shape
    nb = -(-d // BLOCK)
    x = x.float()
    if nb * BLOCK != d:
        x = torch.cat([x, x.new_zeros(n, nb * BLOCK - d)], 1)
    return x.view(n, nb, BLOCK)


def _quantise_plain(x):
    """Values on the 4-bit grid (signed, scaled by 2^-e) and the exponents e, per block."""
    b = _blocks(x)
    amax = b.abs().amax(2)
    e = torch.frexp(amax)[1] - 3                      # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, -127).clamp(-127, 127)
    y = torch.ldexp(b, -e[..., None])
    a = y.abs()
    # steps of 1/2 below 2, 1 below 4, 2 above; round to even multiples of the step
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.copysign(a, y), e


def _encode_plain(x):
    """Packed codes [n, blocks * 16] (low nibble first) and scale bytes [n, blocks]."""
    y, e = _quantise_plain(x)
    a = y.abs()
    code = (torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4))).to(torch.uint8)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    code = code.view(x.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).to(torch.uint8)


def _decode_plain(codes, tiles, n, d):
    nb = -(-d // BLOCK)
    bt = -(-nb // 4)
    s = tiles.view(-1, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, bt * 4)[:n, :nb]
    nib = torch.stack([codes & 15, codes >> 4], 2).view(n, nb, BLOCK)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    y = torch.ldexp(grid[nib.int()], s[..., None].int() - 127)
    return y.reshape(n, nb * BLOCK)[:, :d]


def _encode_run(x):
    y, e = _quantise_plain(x)
    return torch.ldexp(y, e[..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]].to(x.dtype)


def _scores_run(state):
    case, q = state["case"], state["q"]
    y, e = _quantise_plain(q)
    q = torch.ldexp(y, e[..., None]).reshape(q.shape[0], -1)[:, :q.shape[1]]
    s = state["alpha"] * (q @ _decode_plain(state["codes"], state["scales"], case["n"], case["d"]).T)
    if state["bias"] is not None:
        s += state["bias"]
    return s.to(DTYPES[case["out"]])


def _sample_run(state):
    x = state["logits"].double()
    t = state["temperature"].double()[:, None]
    v = x.shape[1]
    top, first = x.max(1, keepdim=True)
    dead = top == -math.inf
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    first = order[:, :1]
    delta = torch.where(x == top, 0.0, (x - top) / torch.where(t > 0, t, 1.0))
    w = torch.exp(delta).masked_fill(x == -math.inf, 0.0)
    ws = w.gather(1, order)
    rank = torch.arange(v, device=x.device)[None]
    keep = torch.ones_like(x, dtype=torch.bool)
    if state["top_k"] is not None:
        k = state["top_k"].long()[:, None]
        keep &= (rank < k) | (k <= 0)
        ws = ws * keep
    if state["top_p"] is not None:
        before = ws.cumsum(1) - ws
        keep &= (before < state["top_p"].double()[:, None] * ws.sum(1, keepdim=True)) | (rank == 0)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    if state["min_p"] is not None:
        kept &= w >= state["min_p"].double()[:, None]
    w = w * kept
    total = w.sum(1, keepdim=True)
    run = w.cumsum(1)
    pick = (run > state["u"][:, None] * total).int().argmax(1, keepdim=True)
    prob = w.gather(1, pick) / total
    pick = torch.where(t > 0, pick, first)
    prob = torch.where(t > 0, prob, 1.0)
    pick = torch.where(dead, -1, pick)
    prob = torch.where(dead, 0.0, prob)
    return {"ids": pick[:, 0].int(), "prob": prob[:, 0].float()}


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        import ivf_quantizer_b200 as q
        if case["op"] == "encode":
            return q.MX4(state["x"]).decode(state["x"].dtype)
        if case["op"] == "scores":
            index = q.MX4.from_codes(state["codes"], state["scales"], case["d"])
            return index.scores(state["q"], alpha=state["alpha"], bias=state["bias"],
                                dtype=DTYPES[case["out"]])
        ids, prob = q.sample_logits(state["logits"], state["u"], temperature=state["temperature"],
                                    top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
        return {"ids": ids, "prob": prob}
    if case["op"] == "encode":
        return _encode_run(state["x"])
    if case["op"] == "scores":
        return _scores_run(state)
    return _sample_run(state)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "encode":
        n, d = case["n"], case["d"]
        code = n * -(-d // BLOCK) * 17
        return {"bytes": 2 * n * d * size[case["dtype"]] + 2 * code, "flops": 0}
    if case["op"] == "scores":
        m, n, d = case["m"], case["n"], case["d"]
        nbytes = m * d * size[case["dtype"]] + n * -(-d // BLOCK) * 17 + m * n * size[case["out"]]
        return {"bytes": nbytes + (4 * n if case["bias"] else 0), "flops": 2 * m * n * d}
    r, v = case["rows"], case["v"]
    params = 12 + 4 * (case["topk"] + case["topp"] + case["minp"])
    return {"bytes": r * (v * size[case["dtype"]] + params + 8), "flops": 2 * r * v}


# ------------------------------------------------------------------ definitions in 64 bits
def _exact_values(x):
    """What the codes of x stand for, from the nearest grid value (ties: even code)."""
    x = x.double()
    n, d = x.shape
    out = torch.empty_like(x)
    mid = torch.tensor([(a + b) / 2 for a, b in zip(GRID, GRID[1:])], device=x.device, dtype=torch.float64)
    grid = torch.tensor(GRID, device=x.device, dtype=torch.float64)
    for b in range(0, d, BLOCK):
        part = x[:, b:b + BLOCK]
        top = part.abs().max(1, keepdim=True)[0]
        e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e)) - 2
        scale = torch.exp2(torch.where(top > 0, e, -127.0).clamp(-127, 127))
        a = (part.abs() / scale).contiguous()
        low = torch.bucketize(a, mid)                   # mid[i-1] < a <= mid[i]
        tie = (low < 7) & (a == mid[low.clamp(max=6)]) & (low % 2 == 1)
        out[:, b:b + BLOCK] = torch.sign(part) * grid[low + tie.long()] * scale
    return out


def _exact_index(codes, tiles, n, d):
    """Row-major values of an index, each byte looked up on its own."""
    nb = -(-d // BLOCK)
    r = torch.arange(n, device=codes.device)[:, None]
    b = torch.arange(nb, device=codes.device)[None]
    at = ((r // 128) * -(-nb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    scale = torch.exp2(tiles[at].double() - 127)
    i = torch.arange(d, device=codes.device)
    nib = (codes[:, i // 2].long() >> (4 * (i % 2))) & 15
    grid = torch.tensor(GRID, device=codes.device, dtype=torch.float64)
    return torch.where(nib > 7, -1.0, 1.0) * grid[nib % 8] * scale[:, i // BLOCK]


def _exact_row(x, u, t, k, p, m):
    if not np.any(x > -np.inf):
        return -1, 0.0
    order = np.lexsort((np.arange(len(x)), -x))         # descending, ties to the lower index
    if t == 0:
        return int(order[0]), 1.0
    w = np.where(x == x.max(), 1.0, np.exp((x - x.max()) / t))
    if k is not None and 0 < k < len(x):
        order = order[:k]
    if p is not None:
        mass = np.cumsum(w[order])
        order = order[:1 + int(np.count_nonzero(mass[:-1] < p * mass[-1]))]
    if m is not None:
        order = order[w[order] >= m]
    order = np.sort(order)
    mass = np.cumsum(w[order])
    j = order[min(int(np.searchsorted(mass, u * mass[-1], side="right")), len(order) - 1)]
    return int(j), float(w[j] / mass[-1])


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "encode":
        x = state["x"]
        at = range(0, x.shape[0], max(1, (1 << 26) // x.shape[1]))
        step = max(1, (1 << 26) // x.shape[1])
        return torch.cat([_exact_values(x[i:i + step]).to(torch.float32) for i in at])
    if case["op"] == "scores":
        n, step = case["n"], max(128, (1 << 26) // case["d"] // 128 * 128)
        q = _exact_values(state["q"])
        out = []
        bt = -(-(-(-case["d"] // BLOCK)) // 4)
        for i in range(0, n, step):
            rows = min(step, n - i)
            y = _exact_index(state["codes"][i:i + rows], state["scales"][i // 128 * bt * 512:], rows, case["d"])
            s = state["alpha"] * (q @ y.T)
            out.append(s if state["bias"] is None else s + state["bias"][i:i + rows].double())
        return torch.cat(out, 1)
    got = {k: state[k].cpu().double().numpy() if state[k] is not None else None
           for k in ("logits", "u", "temperature", "top_k", "top_p", "min_p")}
    ids, prob = [], []
    for i in range(case["rows"]):
        pick = [None if got[k] is None else got[k][i] for k in ("u", "temperature", "top_k", "top_p", "min_p")]
        j, w = _exact_row(got["logits"][i], pick[0], pick[1], None if pick[2] is None else int(pick[2]), *pick[3:])
        ids.append(j)
        prob.append(w)
    return {"ids": torch.tensor(ids, dtype=torch.int32), "prob": torch.tensor(prob, dtype=torch.float64)}
