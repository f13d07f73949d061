"""Cases, plain forms and exact forms of the 8-bit operators.

A matrix in 8 bits is E4M3 codes with one power-of-two scale 2^E per block: 1 x 128 elements along a row
(activations) or 128 x 128 (weights).  E is the smallest integer with 448 * 2^E >= max|a| over the block's finite
elements (at least -127; 0 for a block of zeros), the code is a * 2^-E rounded to nearest-even E4M3, and an
element that is not finite gets the NaN code.  Scales are bytes E + 127, rows of 4 * ceil(columns / 512) bytes
(bytes behind the last block hold 127).

Operators, with ^ for a dequantised matrix:
  quantize   codes and scales of a matrix
  matmul     Y = A^ B^T
  forward    x^ = 1 x 128 blocks of x;  T_p = x V_p;  y_p = s_p (.) (x^ W^_p^T) + T_p U_p^T;
             with a checkpoint it also returns the codes and scales of x and T_p
  backward   from the checkpoint and dy_p:  E_p = dy_p U_p;  g_p = 1 x 128 blocks of s_p (.) dy_p;
             dx = sum_p g_p^ W^_p + E_p V_p^T;  ds_p = sum_m dy_p (.) (x^ W^_p^T);
             dU_p = dy_p^T T_p;  dV_p = x^^T E_p
"""
import math

import torch

own = False

_DEV = "cuda"


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # one token's activations on their way into an 8-bit product
        {"name": "quantize one token", "op": "quantize", "rows": 1, "cols": 1152, "block": 1, "type": "bf16"},
        # the shared gate block of a Gemma-4-31B band, put into 8 bits at load time
        {"name": "quantize gate weight", "op": "quantize", "rows": 21504, "cols": 5376, "block": 128, "type": "bf16"},
        # a band mean as the host decomposition leaves it (fp32), ragged against the blocks
        {"name": "quantize fp32 ragged", "op": "quantize", "rows": 1000, "cols": 4112, "block": 128, "type": "fp32"},
        # a Gemma-3-1B q block against a short prompt already in 8 bits
        {"name": "matmul q 48 tokens", "op": "matmul", "M": 48, "N": 1024, "K": 1152},
        # the Gemma-4-31B o block against a prefill chunk
        {"name": "matmul o prefill", "op": "matmul", "M": 4096, "N": 5376, "K": 8192},
        # Gemma-3-1B q/k/v for one token: the shortest call of a decode step
        {"name": "forward 1b qkv decode", "op": "forward", "M": 1, "K": 1152, "N": "1024,256,256", "r": "16,16,16", "save": False},
        # Gemma-4-31B gate/up for one token: the longest weight stream of a decode step
        {"name": "forward 31b gate/up decode", "op": "forward", "M": 1, "K": 5376, "N": "21504,21504", "r": "256,256", "save": False},
        # Gemma-4-31B down for a batch of 16 decoding sequences
        {"name": "forward 31b down 16", "op": "forward", "M": 16, "K": 21504, "N": "5376", "r": "256", "save": False},
        # ragged stack: odd token count, rows and columns that end inside a block, one projection without a delta
        {"name": "forward ragged 333", "op": "forward", "M": 333, "K": 2000, "N": "1001,264,77", "r": "40,0,8", "save": True},
        # Gemma-4-31B q/k/v over a training batch that keeps its checkpoint
        {"name": "forward 31b qkv save", "op": "forward", "M": 4096, "K": 5376, "N": "8192,4096,4096", "r": "256,256,256", "save": True},
        # Gemma-3-1B gate/up, a small training batch
        {"name": "backward 1b gate/up", "op": "backward", "M": 512, "K": 1152, "N": "4096,4096", "r": "16,16"},
        # Gemma-4-31B q/k/v, the backward of the training batch above
        {"name": "backward 31b qkv", "op": "backward", "M": 4096, "K": 5376, "N": "8192,4096,4096", "r": "256,256,256"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "forward", "forward", "forward", "backward", "backward"])
    while True:
        if op == "quantize":
            c = {"op": op, "rows": _log_int(rng, 1, 21504), "cols": _log_int(rng, 16, 21504, 16), "block": rng.choice([1, 128]),
                 "type": rng.choice(["bf16", "fp32"])}
            if c["rows"] * c["cols"] <= 21504 * 5376:
                return c
            continue
        M, K = _log_int(rng, 1, 4096), _log_int(rng, 64, 21504, 16)
        if op == "matmul":
            c = {"op": op, "M": M, "N": _log_int(rng, 16, 21504), "K": K}
            if M * c["N"] * K <= 4096 * 5376 * 8192:
                return c
            continue
        P = rng.choice([1, 1, 2, 3])
        N = [_log_int(rng, 16, 21504 // P) for _ in range(P)]
        r = [8 * rng.randint(0, 32) for _ in range(P)]
        c = {"op": op, "M": M, "K": K, "N": ",".join(map(str, N)), "r": ",".join(map(str, r))}
        if op == "forward":
            c["save"] = rng.random() < 0.5
        if M * K * sum(N) <= 4096 * 5376 * 16384 and K * sum(N) <= 5376 * 43008:
            return c


def _ints(text):
    return [int(v) for v in str(text).split(",")]


def _scale_pitch(cols):
    return 4 * -(-cols // 512)


def work(case):
    op = case["op"]
    if op == "quantize":
        R, C, b = case["rows"], case["cols"], case["block"]
        return {"bytes": R * C * (3 if case["type"] == "bf16" else 5) + -(-R // b) * _scale_pitch(C), "flops": 0}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 2 * M * N + M * _scale_pitch(K) + -(-N // 128) * _scale_pitch(K), "flops": 2 * M * N * K}
    M, K, N, r = case["M"], case["K"], _ints(case["N"]), _ints(case["r"])
    sc = _scale_pitch(K)
    weights = sum(n * K + -(-n // 128) * sc + 4 * n + 2 * q * (n + K) for n, q in zip(N, r))
    if op == "forward":
        saved = M * K + M * sc + 2 * M * sum(r) if case["save"] else 0
        return {"bytes": 2 * M * K + weights + 2 * M * sum(N) + saved, "flops": sum(2 * M * n * K + 2 * M * q * (n + K) for n, q in zip(N, r))}
    grads = sum(4 * n + 2 * q * (n + K) for n, q in zip(N, r))
    return {"bytes": M * K + M * sc + 2 * M * sum(r) + weights + 2 * M * sum(N) + 2 * M * K + grads,
            "flops": sum(4 * M * n * K + 4 * M * q * (n + K) for n, q in zip(N, r))}


# ------------------------------------------------------------- plain forms ----
def _quantize(a, block):
    """Codes (as E4M3 values) and scale bytes of a fp32 matrix."""
    R, C = a.shape
    RB, CB = -(-R // block), -(-C // 128)
    size = torch.where(torch.isfinite(a), a.abs(), 0.0)
    size = torch.nn.functional.pad(size, (0, CB * 128 - C, 0, RB * block - R))
    top = size.view(RB, block, CB, 128).amax(dim=(1, 3))
    m, e = torch.frexp(top)
    E = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-127), 0)
    codes = torch.ldexp(a, -_spread(E, block, R, C)).to(torch.float8_e4m3fn)
    scales = torch.full((RB, _scale_pitch(C)), 127, dtype=torch.uint8, device=a.device)
    scales[:, :CB] = (E + 127).to(torch.uint8)
    return codes, scales


def _spread(E, block, R, C):
    return E.repeat_interleave(block, 0)[:R].repeat_interleave(128, 1)[:, :C]


def _values(codes, scales, block):
    """The matrix that codes and scales stand for, in fp32."""
    R, C = codes.shape
    E = scales[:, : -(-C // 128)].to(torch.int32) - 127
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), _spread(E, block, R, C))


def _plain_forward(state):
    x, save = state["x"].float(), state["save"]
    codes, scales = _quantize(x, 1)
    xh = _values(codes, scales, 1)
    T = [x @ V.float() if U is not None else None for (_, _, _, U, V) in state["projs"]]
    y = [_plain_projection(xh, t, *p).to(torch.bfloat16) for t, p in zip(T, state["projs"])]
    out = {"y": y}
    if save:
        out.update(codes=codes, scales=scales, T=[t.to(torch.bfloat16) for t in T if t is not None])
    return out


def _plain_projection(xh, t, codes, scales, s, U, V):
    z = s * (xh @ _values(codes, scales, 128).T)
    return z if t is None else z + t @ U.float().T


def _plain_gradients(xh, dy, T, codes, scales, s, U, V):
    """One projection's part of dx, and ds, dU, dV."""
    W = _values(codes, scales, 128)
    dy = dy.float()
    g = _values(*_quantize(s * dy, 1), 1)
    dx, ds = g @ W, (dy * (xh @ W.T)).sum(0)
    if U is None:
        return dx, ds, None, None
    E = dy @ U.float()
    return dx + E @ V.float().T, ds, (dy.T @ T.float()).to(torch.bfloat16), (xh.T @ E).to(torch.bfloat16)


def _plain_backward(state):
    xh = _values(state["codes"], state["scales"], 1)
    got = [_plain_gradients(xh, dy, T, *p) for dy, T, p in zip(state["dy"], state["T"], state["projs"])]
    return _gradients(sum(g[0] for g in got).to(torch.bfloat16), [g[1:] for g in got])


def _gradients(dx, per):
    return {"dx": dx, "ds": [g[0] for g in per], "dU": [g[1] for g in per if g[1] is not None], "dV": [g[2] for g in per if g[2] is not None]}


# ---------------------------------------------------------------- prepare ----
def _activations(g, M, K):
    """Unit-variance tokens with a few channels twenty times as large, as the residual stream of a trained model has."""
    x = torch.randn(M, K, generator=g, device=_DEV)
    big = torch.rand(K, generator=g, device=_DEV) < 0.004
    return torch.where(big, 20 * x, x).to(torch.bfloat16)


def _weight(g, N, K):
    codes, scales = _quantize((0.02 * torch.randn(N, K, generator=g, device=_DEV)).to(torch.bfloat16).float(), 128)
    return codes.view(torch.uint8), scales


def _bundle(g, N, K, r):
    codes, scales = _weight(g, N, K)
    s = 0.9 + 0.2 * torch.rand(N, generator=g, device=_DEV)
    U = (0.02 * torch.randn(N, r, generator=g, device=_DEV)).to(torch.bfloat16) if r else None
    V = (0.02 * torch.randn(K, r, generator=g, device=_DEV)).to(torch.bfloat16) if r else None
    return codes, scales, s, U, V


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    state = dict(case)
    op = case["op"]
    if op == "quantize":
        a = _activations(g, case["rows"], case["cols"]) if case["block"] == 1 else 0.02 * torch.randn(case["rows"], case["cols"], generator=g, device=_DEV)
        state["a"] = a.to(torch.bfloat16 if case["type"] == "bf16" else torch.float32)
        return state
    M, K = case["M"], case["K"]
    x = _activations(g, M, K)
    if op == "matmul":
        codes, scales = _quantize(x.float(), 1)
        state.update(A=(codes.view(torch.uint8), scales), B=_weight(g, case["N"], K))
        return state
    N, r = _ints(case["N"]), _ints(case["r"])
    state["projs"] = [_bundle(g, n, K, q) for n, q in zip(N, r)]
    if op == "forward":
        state["x"] = x
        if own and not case["save"]:
            import linear_wl_forward_b200 as wl

            # a decode program keeps one handle per call of its step
            state["handle"] = wl.prepare_stacked_fp8(x, state["projs"])
        return state
    codes, scales = _quantize(x.float(), 1)
    state.update(codes=codes.view(torch.uint8), scales=scales)
    state["T"] = [(x.float() @ V.float()).to(torch.bfloat16) if V is not None else None for (_, _, _, _, V) in state["projs"]]
    state["dy"] = [(1e-3 * torch.randn(M, n, generator=g, device=_DEV)).to(torch.bfloat16) for n in N]
    return state


# -------------------------------------------------------------------- run ----
def run(state):
    op = state["op"]
    if own:
        import linear_wl_forward_b200 as wl

        if op == "quantize":
            codes, scales = wl.quantize_fp8(state["a"], block_rows=state["block"])
            return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales}
        if op == "matmul":
            return wl.matmul_fp8(state["A"], state["B"])
        if op == "forward":
            if not state["save"]:
                return {"y": state["handle"]()}
            y, ckpt = wl.stacked_forward_fp8(state["x"], state["projs"], checkpoint=True)
            return {"y": y, "codes": ckpt.codes.view(torch.float8_e4m3fn), "scales": ckpt.scales, "T": [t for t in ckpt.T if t is not None]}
        ckpt = wl.Fp8Checkpoint(state["codes"], state["scales"], state["T"])
        dx, per = wl.stacked_backward_fp8(ckpt, state["dy"], state["projs"])
        return _gradients(dx, per)
    if op == "quantize":
        codes, scales = _quantize(state["a"].float(), state["block"])
        return {"codes": codes, "scales": scales}
    if op == "matmul":
        return (_values(*state["A"], 1) @ _values(*state["B"], 128).T).to(torch.bfloat16)
    return _plain_forward(state) if op == "forward" else _plain_backward(state)


# ------------------------------------------------------------------ exact ----
def _e4m3(v):
    """v (fp64) on the E4M3 grid: steps of 2^(exponent - 3), exponent at least -6, ties to even; what is not finite stays so."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.where(torch.isfinite(v), torch.round(v / step) * step, math.nan)


def _exact_blocks(a, block):
    """E4M3 values and 2^E per element of a fp64 matrix, E by comparing with 448 * 2^E."""
    R, C = a.shape
    RB, CB = -(-R // block), -(-C // 128)
    full = torch.zeros(RB * block, CB * 128, dtype=torch.float64, device=a.device)
    full[:R, :C] = torch.where(torch.isfinite(a), a, 0.0).abs()
    top = torch.stack([b.reshape(RB, -1).amax(1) for b in full.view(RB, block, CB * 128).split(128, dim=2)], dim=1)
    E = torch.full_like(top, -127.0)
    for e in range(-126, 122):  # one step up for every limit that the block is above
        E += (top > 448.0 * 2.0 ** (e - 1)).double()
    E = torch.where(top == 0, 0.0, E)
    per = torch.exp2(E)[:, None, :, None].expand(RB, block, CB, 128).reshape(RB * block, CB * 128)[:R, :C]
    return _e4m3(a / per), per


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        v, per = _exact_blocks(state["a"].double(), case["block"])
        return {"codes": v, "scales": None}
    if op == "matmul":
        (a, sa), (b, sb) = state["A"], state["B"]
        return _exact_values(a, sa, 1) @ _exact_values(b, sb, 128).mT
    projs = state["projs"]
    if op == "forward":
        x = state["x"].double()
        v, per = _exact_blocks(x, 1)
        y, T = [], []
        for codes, scales, s, U, V in projs:
            z = (v * per) @ _exact_values(codes, scales, 128).mT * s.double()
            if U is not None:
                T.append(x @ V.double())
                z += T[-1] @ U.double().mT
            y.append(z)
        return {"y": y, "codes": v, "scales": None, "T": T} if case["save"] else {"y": y}
    xh = _exact_values(state["codes"], state["scales"], 1)
    dx, ds, dU, dV = torch.zeros_like(xh), [], [], []
    for (codes, scales, s, U, V), dy, T in zip(projs, state["dy"], state["T"]):
        W, d = _exact_values(codes, scales, 128), dy.double()
        v, per = _exact_blocks(d * s.double(), 1)
        dx += (v * per) @ W
        ds.append(torch.einsum("mn,mn->n", d, xh @ W.mT))
        if U is not None:
            E = d @ U.double()
            dx += E @ V.double().mT
            dU.append(d.mT @ T.double())
            dV.append(xh.mT @ E)
    return {"dx": dx, "ds": ds, "dU": dU, "dV": dV}


def _exact_values(codes, scales, block):
    """Codes and scales read by their bits: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7F is NaN."""
    c = codes.to(torch.int32)
    sign, e, m = 1.0 - 2.0 * (c >> 7).double(), (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    v = sign * torch.where((c & 127) == 127, math.nan, v)
    R, C = codes.shape
    rows, cols = torch.arange(R, device=c.device) // block, torch.arange(C, device=c.device) // 128
    return v * torch.exp2(scales.double() - 127)[rows][:, cols]
