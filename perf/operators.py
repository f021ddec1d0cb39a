"""Cases of the 8-bit projection operators: the residual's addition with RMSNorm and an e4m3 output
(csa_add_norm_quant), the e4m3 storage of a weight in 128 x 128 blocks (csa_quantize_weight) and the matrix product over
such operands (csa_fp8_proj).

8-bit storage, everywhere: a block of values shares the float32 scale max(amax / 448, 2^-126); a value's e4m3 code is
value / scale rounded to nearest even. Codes are returned as float8_e4m3fn numbers beside their scales (a code times its
scale is the value that it stands for)."""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 2.0 ** -126
EPS = 1e-6


# ---------------------------------------------------------------- cases

def _norm(rows, d, dtype="bf16", residual=True, normalise=True, y=False, **more):
    return {"op": "norm", "rows": rows, "d": d, "dtype": dtype, "residual": residual, "normalise": normalise, "y": y, **more}


def _weight(N, K, dtype="bf16", **more):
    return {"op": "weight", "N": N, "K": K, "dtype": dtype, **more}


def _proj(M, N, K, out="bf16", groups=1, **more):
    return {"op": "proj", "M": M, "N": N, "K": K, "out": out, "groups": groups, **more}


def listed():
    return [
        # one decode step of 8 sequences, hidden width 4096: the launch's latency is all of it
        _norm(8, 4096, name="norm_decode_8"),
        # the hidden states of a long prefill, before the layer's projections
        _norm(65536, 4096, name="norm_prefill_65536"),
        # float32 activations of a ragged batch, a last group of 16 channels, the normed values wanted too
        _norm(1537, 2064, "f32", residual=False, y=True, name="norm_f32_ragged"),
        # the outputs of 64 attention heads of width 512 on their way to the grouped output projection
        _norm(4096, 32768, residual=False, normalise=False, name="quant_heads_4096"),
        # storing the query up-projection (latent 1024 -> 64 heads of 512), as done once for each layer of a model
        _weight(32768, 1024, name="weight_query"),
        # a float32 weight whose edge blocks are cut on both sides
        _weight(1000, 1040, "f32", name="weight_f32_ragged"),
        # one token through the query's down-projection: latency
        _proj(1, 1024, 4096, name="proj_decode_1"),
        # a decode step of 8 sequences through the query up-projection: the weight's bytes
        _proj(8, 32768, 1024, name="proj_decode_8"),
        # a short ragged prompt, float32 results, cut tiles on every side
        _proj(333, 1000, 2064, "f32", name="proj_f32_ragged"),
        # one of the compressor's projections for a prompt of 4096 tokens
        _proj(4096, 512, 2048, name="proj_kv_4096"),
        # indexer queries of 64 heads of 128, written in 8 bits with a scale for each head
        _proj(32768, 8192, 1024, "e4m3", name="proj_index_queries"),
        # the grouped output projection: 8 groups of 8 heads of 512, 1024 features each
        _proj(16384, 1024, 4096, groups=8, name="proj_grouped_out"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "weight", "proj", "proj", "proj"])
    if kind == "norm":
        d = 16 * _log(rng, 4, 2048)
        rows = _log(rng, 1, max(2, min(65536, (1 << 27) // d)))
        return _norm(rows, d, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.75, rng.random() < 0.3)
    if kind == "weight":
        return _weight(_log(rng, 1, 16384), 16 * _log(rng, 4, 256), rng.choice(["bf16", "f32"]))
    M = _log(rng, 1, 16384)
    out = rng.choice(["bf16", "bf16", "f32", "e4m3"])
    if rng.random() < 0.2:
        return _proj(M, BLOCK * rng.randint(1, 8), BLOCK * rng.randint(1, 16), out, rng.randint(2, 8))
    N = 16 * _log(rng, 1, 512) if out == "e4m3" else _log(rng, 1, 8192)
    return _proj(M, N, 16 * _log(rng, 4, 256), out)


# ---------------------------------------------------------------- inputs

def _pad(n):
    return -(-n // BLOCK) * BLOCK


def _groups_of_row(y):
    """y [rows, d] float32 -> [rows, ceil(d / 128), 128], zeros behind the last channel."""
    rows, d = y.shape
    if d % BLOCK:
        y = torch.nn.functional.pad(y, (0, _pad(d) - d))
    return y.reshape(rows, -1, BLOCK)


def _rows_to_e4m3(y):
    """Codes [rows, d] and scales [rows, ceil(d / 128)] of float32 rows."""
    g = _groups_of_row(y)
    scale = (g.abs().amax(-1) / 448.0).clamp_min(TINY)
    codes = (g / scale[:, :, None]).clamp(-448.0, 448.0).to(F8)
    return codes.reshape(y.shape[0], -1)[:, :y.shape[1]].contiguous(), scale


def _blocks_to_e4m3(w):
    """Codes [N, K] and scales [ceil(N / 128), ceil(K / 128)] of a float32 weight."""
    N, K = w.shape
    p = torch.nn.functional.pad(w, (0, _pad(K) - K, 0, _pad(N) - N)).reshape(_pad(N) // BLOCK, BLOCK, -1, BLOCK)
    scale = (p.abs().amax((1, 3)) / 448.0).clamp_min(TINY)
    codes = (p / scale[:, None, :, None]).clamp(-448.0, 448.0).to(F8)
    return codes.reshape(_pad(N), -1)[:N, :K].contiguous(), scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = dict(case)
    if case["op"] == "norm":
        rows, d, dt = case["rows"], case["d"], TYPES[case["dtype"]]
        # hidden states: some channels carry far larger values than the rest, and so do some tokens
        x = normal(rows, d).mul_((0.7 * normal(d)).exp_()).mul_((0.4 * normal(rows, 1)).exp_())
        s["x"] = x.to(dt)
        del x
        s["residual"] = s["total"] = s["gamma"] = s["y_out"] = None
        if case["residual"]:
            s["residual"] = normal(rows, d).mul_(2.0).to(dt)
            s["total"] = torch.empty(rows, d, device=DEV, dtype=dt)
        if case["normalise"]:
            s["gamma"] = normal(d).mul_(0.1).add_(1.0)
        if case["y"]:
            s["y_out"] = torch.empty(rows, d, device=DEV, dtype=dt)
        s["codes"] = torch.empty(rows, d, device=DEV, dtype=F8)
        s["scale"] = torch.empty(rows, _pad(d) // BLOCK, device=DEV)
    elif case["op"] == "weight":
        N, K = case["N"], case["K"]
        s["W"] = normal(N, K).mul_(0.02).mul_((0.3 * normal(N, 1)).exp_()).to(TYPES[case["dtype"]])
        s["codes"] = torch.empty(N, K, device=DEV, dtype=F8)
        s["scale"] = torch.empty(_pad(N) // BLOCK, _pad(K) // BLOCK, device=DEV)
    else:
        M, N, K, G = (case[k] for k in ("M", "N", "K", "groups"))
        s["A"], s["A_scale"] = _rows_to_e4m3(normal(M, G * K).mul_((0.5 * normal(M, 1)).exp_()))
        s["W"], s["W_scale"] = _blocks_to_e4m3(normal(G * N, K).mul_(0.02))
        s["out_scale"] = None
        if case["out"] == "e4m3":
            s["result"] = torch.empty(M, G * N, device=DEV, dtype=F8)
            s["out_scale"] = torch.empty(M, _pad(G * N) // BLOCK, device=DEV)
        else:
            s["result"] = torch.empty(M, G * N, device=DEV, dtype=TYPES[case["out"]])
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "weight": _plain_weight, "proj": _plain_proj}[state["op"]](state)


def _own(s):
    from long_context_sparse_07_b200 import abi
    if s["op"] == "norm":
        abi.csa_add_norm_quant(s["x"], s["residual"], s["gamma"], normalise=s["normalise"], eps=EPS, total=s["total"],
                               y=s["y_out"], codes=s["codes"], scale=s["scale"])
        return {"total": s["total"], "y": s["y_out"], "codes": s["codes"], "scale": s["scale"]}
    if s["op"] == "weight":
        abi.csa_quantize_weight(s["W"], s["codes"], s["scale"])
        return {"codes": s["codes"], "scale": s["scale"]}
    abi.csa_fp8_proj(s["A"], s["A_scale"], s["W"], s["W_scale"], s["result"], s["out_scale"], groups=s["groups"])
    return {"result": s["result"], "scale": s["out_scale"]}


def _plain_norm(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    total = v.to(s["x"].dtype) if s["residual"] is not None else None
    if s["normalise"]:
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * s["gamma"]
    codes, scale = _rows_to_e4m3(v)
    return {"total": total, "y": v.to(s["x"].dtype) if s["y"] else None, "codes": codes, "scale": scale}


def _plain_weight(s):
    codes, scale = _blocks_to_e4m3(s["W"].float())
    return {"codes": codes, "scale": scale}


def _row_values(codes, scale):
    """The float32 values of e4m3 rows with a scale for each 128 channels."""
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _block_values(codes, scale):
    N, K = codes.shape
    return codes.float() * scale.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _plain_proj(s):
    M, N, K, G = (s[k] for k in ("M", "N", "K", "groups"))
    a = _row_values(s["A"], s["A_scale"]).reshape(M, G, K).transpose(0, 1)
    w = _block_values(s["W"], s["W_scale"]).reshape(G, N, K)
    out = torch.matmul(a, w.transpose(1, 2)).transpose(0, 1).reshape(M, G * N)
    if s["out"] == "e4m3":
        codes, scale = _rows_to_e4m3(out)
        return {"result": codes, "scale": scale}
    return {"result": out.to(TYPES[s["out"]]), "scale": None}


# ---------------------------------------------------------------- work, and values in 64 bits

def work(case):
    b = {"bf16": 2, "f32": 4, "e4m3": 1}
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        wide = (1 + 2 * case["residual"] + case["y"]) * b[case["dtype"]]
        return {"bytes": rows * (d * (wide + 1) + 4 * (_pad(d) // BLOCK)) + 4 * d * case["normalise"], "flops": 8 * rows * d}
    if case["op"] == "weight":
        N, K = case["N"], case["K"]
        return {"bytes": N * K * (b[case["dtype"]] + 1) + 4 * (_pad(N) // BLOCK) * (_pad(K) // BLOCK), "flops": 3 * N * K}
    M, N, K, G = (case[k] for k in ("M", "N", "K", "groups"))
    kb = _pad(K) // BLOCK
    out = M * G * N * b[case["out"]] + (4 * M * (_pad(G * N) // BLOCK) if case["out"] == "e4m3" else 0)
    return {"bytes": G * (M * K + N * K + 4 * M * kb + 4 * (_pad(N) // BLOCK) * kb) + out, "flops": 2 * M * N * K * G}


def _exact_groups(v):
    """Codes before their rounding, and scales, of float64 rows: one slice of 128 channels after the other."""
    codes, scales = [], []
    for lo in range(0, v.shape[1], BLOCK):
        part = v[:, lo:lo + BLOCK]
        a = torch.maximum(part.abs().max(dim=1, keepdim=True).values / 448, torch.full_like(part[:, :1], TINY))
        codes.append(part / a)
        scales.append(a)
    return torch.cat(codes, 1), torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        parts = []
        step = max(1, (1 << 26) // case["d"])
        for lo in range(0, case["rows"], step):
            v = s["x"][lo:lo + step].double()
            total = None
            if case["residual"]:
                v = total = v + s["residual"][lo:lo + step].double()
            if case["normalise"]:
                v = v / torch.sqrt((v * v).sum(1, keepdim=True) / case["d"] + EPS) * s["gamma"].double()
            codes, scale = _exact_groups(v)
            parts.append((total, v if case["y"] else None, codes, scale))
        total, y, codes, scale = (None if p[0] is None else torch.cat(p) for p in zip(*parts))
        return {"total": total, "y": y, "codes": codes, "scale": scale}
    if case["op"] == "weight":
        w = s["W"].double()
        N, K = w.shape
        codes, scale = torch.empty_like(w), torch.empty_like(s["scale"], dtype=torch.float64)
        for i in range(scale.shape[0]):
            rows = w[i * BLOCK:(i + 1) * BLOCK]
            for j in range(scale.shape[1]):
                part = rows[:, j * BLOCK:(j + 1) * BLOCK]
                a = torch.clamp(part.abs().max() / 448, min=TINY)
                scale[i, j] = a
                codes[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = part / a
        return {"codes": codes, "scale": scale}
    M, N, K, G = (case[k] for k in ("M", "N", "K", "groups"))
    kb = _pad(K) // BLOCK
    out = torch.zeros(M, G * N, device=DEV, dtype=torch.float64)
    row_block = torch.arange(G * N, device=DEV) // BLOCK
    for g in range(G):
        cols, rows = slice(g * N, (g + 1) * N), row_block[g * N:(g + 1) * N]
        a = s["A"][:, g * K:(g + 1) * K].to(torch.float64)
        w = s["W"][cols].to(torch.float64)
        for j in range(kb):
            k = slice(j * BLOCK, min(K, (j + 1) * BLOCK))
            a[:, k] *= s["A_scale"][:, g * kb + j, None].double()
            w[:, k] *= s["W_scale"][rows, j, None].double()
        out[:, cols] = a @ w.T
    if case["out"] == "e4m3":
        codes, scale = _exact_groups(out)
        return {"result": codes, "scale": scale}
    return {"result": out, "scale": None}
