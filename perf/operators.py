"""What the operators around a gated feed-forward block with quantized weights cost, and what they compute.

Five passes, each a call or two of the library:

* ``gated``: h = act(x Wg^T) * (x Wu^T), the layer's rows being the gate rows and then the up rows.
* ``step``: the same for training (g and u are kept in 8 bits), then its backward pass from the gradient of h.
* ``backward``: that backward pass from a kept checkpoint: dx = dg Wg + du Wu, and (dg | du) where wanted.
* ``dx``: dx = dy W, the input gradient of one quantized layer.
* ``checkpoint``: an activation to 8 bits with a power-of-two scale per 16 values, and back.

``run`` computes them with elementary torch operations where ``own`` is false and calls the library where
it is true.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math

import torch

own = False

ACTS = ("silu", "gelu_tanh", "gelu")
FORMATS = (("int4", 0, 0), ("int6", 0, 0), ("int6p", 0, 0), ("affine", 2, 64), ("affine", 4, 32), ("affine", 4, 64),
           ("affine", 8, 64), ("affine", 8, 128))


def _case(name, op, fmt, M, N, K, act="silu", bits=0, group=0, dgu=False):
    return {"name": name, "op": op, "fmt": fmt, "bits": bits, "group": group, "M": M, "N": N, "K": K, "act": act,
            "dgu": dgu}


def listed():
    return [
        # one token through a small block: the call's latency
        _case("gated_int4_m1_small", "gated", "int4", 1, 2048, 2048),
        # one token of decoding through a wide block: the weights' bytes
        _case("gated_int4_m1_wide", "gated", "int4", 1, 27648, 5120),
        # a decoding batch on the 6-bit format
        _case("gated_int6_m4", "gated", "int6", 4, 27648, 5120, "gelu_tanh"),
        # a prompt: the tensor cores
        _case("gated_int4_m2048", "gated", "int4", 2048, 27648, 5120),
        # a fine-tuning step through frozen weights, and one with sizes that fill no tile
        _case("step_int4_m2048", "step", "int4", 2048, 27648, 5120),
        _case("step_int6_ragged", "step", "int6", 77, 2006, 768, "gelu"),
        # the backward pass alone, of a long batch, and of a short one with the gradients of both projections
        _case("backward_int4_m4096", "backward", "int4", 4096, 27648, 5120),
        _case("backward_affine2_m129", "backward", "affine", 129, 14336, 4096, "gelu_tanh", 2, 64, True),
        # the down projection's input gradient for a batch, and for a few tokens
        _case("dx_int4_m2048", "dx", "int4", 2048, 5120, 27648),
        _case("dx_affine8_m5", "dx", "affine", 5, 4096, 14336, "silu", 8, 64),
        # a layer's activation kept for the backward pass: a long batch, and a few odd rows
        _case("checkpoint_8192x5120", "checkpoint", "none", 8192, 0, 5120),
        _case("checkpoint_33x1003", "checkpoint", "none", 33, 0, 1003),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("gated", "gated", "step", "backward", "dx", "checkpoint"))
    if op == "checkpoint":
        return {"op": op, "fmt": "none", "bits": 0, "group": 0, "M": _log_uniform(rng, 1, 8192), "N": 0,
                "K": _log_uniform(rng, 16, 5120), "act": "silu", "dgu": False}
    fmt, bits, group = rng.choice(FORMATS)
    unit = max(64, group) if fmt == "affine" else 256
    K = unit * _log_uniform(rng, 1, 14336 // unit)
    half = _log_uniform(rng, 8, 13824)
    N = half if op == "dx" else 2 * half
    most = 2048 * 27648 * 5120 // (1 if op == "step" else 2)
    M = _log_uniform(rng, 1, max(1, min(4096, most // (N * K))))
    if op == "gated" and rng.random() < 0.4:  # decoding batches
        M = rng.randint(1, 32)
    return {"op": op, "fmt": fmt, "bits": bits, "group": group, "M": M, "N": N, "K": K, "act": rng.choice(ACTS),
            "dgu": op == "backward" and rng.random() < 0.5}


# ---- inputs ------------------------------------------------------------------------------------------------

def _row_bytes(fmt, bits, group, K):
    """Bytes a row of the packed codes, group metadata and steps."""
    if fmt == "int4":
        return K // 2, K // 16, K // 64
    if fmt in ("int6", "int6p"):
        return 3 * K // 4, K // 16, K // 128
    return K * bits // 8, 4 * K // group, 0


def _weights(case, r):
    """A packed layer as its loader leaves it on the GPU: codes, group metadata and steps as bytes."""
    fmt, bits, group, N, K = case["fmt"], case["bits"], case["group"], case["N"], case["K"]
    cb, gb, sb = _row_bytes(fmt, bits, group, K)
    u8 = dict(dtype=torch.uint8, device="cuda", generator=r)
    codes = torch.randint(0, 256, (N, cb), **u8)
    uniform = lambda shape, lo, hi: torch.rand(shape, device="cuda", generator=r) * (hi - lo) + lo  # noqa: E731
    if fmt == "int4":
        gmeta = torch.randint(0, 256, (N, gb), **u8)
        steps = torch.stack((uniform((N, K // 256), 2 ** -14, 2 ** -13), uniform((N, K // 256), 2 ** -6, 2 ** -5)), -1)
        steps = steps.half().view(torch.uint8)
    elif fmt in ("int6", "int6p"):
        gmeta = torch.randint(1, 256, (N, gb), **u8)  # int8 scale codes; -128 does not occur in a packed layer
        gmeta[gmeta == 128] = 127
        steps = uniform((N, K // 256), 2 ** -14, 2 ** -13).half().view(torch.uint8)
    else:
        top = float(2 ** bits - 1)
        s = uniform((N, K // group), 0.05, 0.35) / top
        gmeta = torch.stack((s, -s * top * uniform((N, K // group), 0.35, 0.65)), -1).bfloat16().view(torch.uint8)
        steps = torch.zeros(16, dtype=torch.uint8, device="cuda")
    return codes.reshape(-1), gmeta.reshape(-1), steps.reshape(-1)


def prepare(case, seed):
    r = torch.Generator("cuda").manual_seed(seed)
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    normal = lambda rows, cols, s: (torch.randn((rows, cols), device="cuda", generator=r) * s).bfloat16()  # noqa: E731
    state = dict(case)
    if op == "checkpoint":  # rows of unlike magnitude, as the tokens of a batch have
        state["x"] = (torch.randn((M, K), device="cuda", generator=r)
                      * torch.exp(torch.randn((M, 1), device="cuda", generator=r))).bfloat16()
        return state
    state["codes"], state["gmeta"], state["steps"] = _weights(case, r)
    if op in ("gated", "step"):
        state["x"] = normal(M, K, 20.0 / math.sqrt(K))
    if op in ("step", "backward"):
        state["dh"] = normal(M, N // 2, 1e-3)
    if op == "backward":  # the forward pass's checkpoint of (g | u): a row of F values for each token and half
        state["saved"] = _save8(torch.randn((2 * M, N // 2), device="cuda", generator=r) * 2.0)
    if op == "dx":
        state["dy"] = normal(M, N, 1e-3)
    return state


# ---- the plain form ----------------------------------------------------------------------------------------

def _save8(v):
    """fp32 rows -> (codes int8 [rows][padded], exponents uint8 [rows][padded / 16])."""
    rows, cols = v.shape
    v = torch.nn.functional.pad(v, (0, -cols % 16)).reshape(rows, -1, 16)
    key = (v.abs().amax(-1).view(torch.int32) + 0x10000) >> 23
    e = (key - 6).clamp(min=1)
    codes = torch.round(v * ((254 - e) << 23).view(torch.float32)[..., None])
    e = torch.where(key >= 255, 255, e)
    codes = torch.where((key >= 255)[..., None], 0.0, codes)
    return codes.to(torch.int8).reshape(rows, -1), e.to(torch.uint8)


def _restore8(saved, cols):
    codes, e = saved
    scale = (e.int() << 23).view(torch.float32)
    scale = torch.where(e == 255, math.nan, scale)
    v = codes.reshape(*e.shape, 16).float() * scale[..., None]
    return v.reshape(e.shape[0], -1)[:, :cols]


def _dequant(s):
    """The packed layer as fp32 [N][K]."""
    fmt, bits, group, N, K = s["fmt"], s["bits"], s["group"], s["N"], s["K"]
    codes = s["codes"].reshape(N, -1)
    if fmt == "int4":
        q = torch.stack((codes & 15, codes >> 4), -1).reshape(N, K // 256, 8, 32).float()
        gm = s["gmeta"].reshape(N, K // 256, 8, 2, 1).float()
        st = s["steps"].view(torch.float16).reshape(N, K // 256, 1, 2, 1).float()
        scale, zero = gm[..., 0, :] * st[..., 0, :], gm[..., 1, :] * st[..., 1, :]
        return ((q - zero) * scale).reshape(N, K)
    if fmt in ("int6", "int6p"):
        if fmt == "int6":
            b = codes.reshape(N, K // 4, 3).int()
            unit = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
            q = torch.stack([(unit >> (6 * i)) & 63 for i in range(4)], -1)
        else:
            b = codes.reshape(N, K // 256, 192)
            lo = torch.stack((b[..., :128] & 15, b[..., :128] >> 4), -1).reshape(N, K // 256, 256)
            hi = torch.stack([(b[..., 128:] >> (2 * i)) & 3 for i in range(4)], -1).reshape(N, K // 256, 256)
            q = (lo | (hi << 4)).int()
        q = ((q ^ 32) - 32).reshape(N, K // 256, 16, 16).float()
        sc = s["gmeta"].view(torch.int8).reshape(N, K // 256, 16, 1).float()
        return (q * (sc * s["steps"].view(torch.float16).reshape(N, K // 256, 1, 1).float())).reshape(N, K)
    per = 8 // bits
    q = torch.stack([(codes >> (bits * i)) & (2 ** bits - 1) for i in range(per)], -1).reshape(N, K // group, group).float()
    gm = s["gmeta"].view(torch.bfloat16).reshape(N, K // group, 2, 1).float()
    return (q * gm[:, :, 0] + gm[:, :, 1]).reshape(N, K)


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
    return g * p, p + g * torch.exp(-0.5 * g * g) * math.sqrt(0.5 / math.pi)


def _plain_backward(s, w, saved):
    F = s["N"] // 2
    v = _restore8(saved, F).reshape(s["M"], 2, F)
    a, d = _act(v[:, 0], s["act"])
    dh = s["dh"].float()
    dgu = torch.cat((dh * v[:, 1] * d, dh * a), 1)
    out = {"dx": (dgu @ w).bfloat16()}
    if s["dgu"]:
        out["dgu"] = dgu.bfloat16()
    return out


def _plain(s):
    op = s["op"]
    if op == "checkpoint":
        return {"restored": _restore8(_save8(s["x"].float()), s["K"]).bfloat16()}
    w = _dequant(s)
    if op == "dx":
        return {"dx": (s["dy"].float() @ w).bfloat16()}
    if op == "backward":
        return _plain_backward(s, w, s["saved"])
    F = s["N"] // 2
    gu = s["x"].float() @ w.T
    out = {"h": (_act(gu[:, :F], s["act"])[0] * gu[:, F:]).bfloat16()}
    if op == "step":
        out.update(_plain_backward(s, w, _save8(gu.reshape(-1, F))))
    return out


# ---- the library's calls -----------------------------------------------------------------------------------

def _buffers(s, ql):
    """What a program keeps from call to call: the layer's description, outputs and workspaces."""
    M, N, K, op = s["M"], s["N"], s["K"], s["op"]
    bf = lambda r, c: torch.empty((r, c), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if op == "checkpoint":
        return {"saved": ql.alloc_saved8(M, K), "restored": bf(M, K)}
    d = ql.Desc(s["fmt"], N, K, s["bits"], s["group"])
    b = {"desc": d, "w": (s["codes"], s["gmeta"], s["steps"])}
    if op in ("gated", "step"):
        b["h"] = bf(M, N // 2)
        b["ws"] = ql.alloc_gated_workspace(d, M)
    if op != "gated":
        b["dx"] = bf(M, K)
        b["ws_dx"] = ql.alloc_gemm_dx_workspace(d, M)
    if op == "step":
        b["saved"] = ql.alloc_saved8(2 * M, N // 2)
    if s["dgu"]:
        b["dgu"] = bf(M, N)
    return b


def _own(s):
    import int6_quantized_linear_b200 as ql
    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _buffers(s, ql)
    M, op = s["M"], s["op"]
    if op == "checkpoint":
        ql.qlinear_save8(s["x"], M, s["K"], b["saved"])
        ql.qlinear_restore8(b["saved"], M, s["K"], b["restored"])
        return {"restored": b["restored"]}
    if op == "gated":
        ql.qlinear_gated(b["desc"], *b["w"], s["x"], M, s["act"], b["h"], workspace=b["ws"])
        return {"h": b["h"]}
    if op == "dx":
        ql.qlinear_gemm_dx(b["desc"], *b["w"], s["dy"], M, b["dx"], workspace=b["ws_dx"])
        return {"dx": b["dx"]}
    out = {}
    saved = s.get("saved")
    if op == "step":
        saved = b["saved"]
        ql.qlinear_gated(b["desc"], *b["w"], s["x"], M, s["act"], b["h"], saved=saved, workspace=b["ws"])
        out["h"] = b["h"]
    ql.qlinear_gated_backward(b["desc"], *b["w"], saved, s["dh"], M, s["act"], b["dx"], dgu=b.get("dgu"),
                              workspace=b["ws_dx"])
    out["dx"] = b["dx"]
    if s["dgu"]:
        out["dgu"] = b["dgu"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    if op == "checkpoint":  # the activation read, its codes and exponents written and read, the restored one written
        return {"bytes": M * K * 4 + 2 * M * -(-K // 16) * 17, "flops": 0}
    packed = N * sum(_row_bytes(case["fmt"], case["bits"], case["group"], K))
    product = 2 * M * N * K
    if op == "gated":
        return {"bytes": packed + 2 * M * K + M * N, "flops": product}
    if op == "dx":
        return {"bytes": packed + 2 * M * N + 2 * M * K, "flops": product}
    if op == "step":  # x, dh in; h, dx out
        return {"bytes": packed + 4 * M * K + 2 * M * N, "flops": 2 * product}
    saved = 2 * M * -(-N // 32) * 17
    return {"bytes": packed + saved + M * N + 2 * M * K + (2 * M * N if case["dgu"] else 0), "flops": product}


# ---- the definitions in 64 bits ----------------------------------------------------------------------------

def _fields(codes, K, bits):
    """Fields of `bits` bits, lowest first, of rows of little-endian bytes."""
    at = torch.arange(K, device=codes.device) * bits
    lo = codes[:, at // 8].int()
    hi = codes[:, torch.clamp(at // 8 + 1, max=codes.shape[1] - 1)].int()
    return ((lo | (hi << 8)) >> (at % 8).int()) & (2 ** bits - 1)


def _weights64(s, n0, n1):
    """Rows n0 .. n1 - 1 of the layer."""
    fmt, bits, group, N, K = s["fmt"], s["bits"], s["group"], s["N"], s["K"]
    codes, gm = s["codes"].reshape(N, -1)[n0:n1], s["gmeta"].reshape(N, -1)[n0:n1]
    k = torch.arange(K, device="cuda")
    if fmt == "affine":
        m = gm.contiguous().view(torch.bfloat16).double()
        return _fields(codes, K, bits) * m[:, 2 * (k // group)] + m[:, 2 * (k // group) + 1]
    st = s["steps"].reshape(N, -1)[n0:n1].contiguous().view(torch.float16).double()
    if fmt == "int4":
        scale = gm[:, 2 * (k // 32)].double() * st[:, 2 * (k // 256)]
        zero = gm[:, 2 * (k // 32) + 1].double() * st[:, 2 * (k // 256) + 1]
        return (_fields(codes, K, 4) - zero) * scale
    if fmt == "int6":
        q = _fields(codes, K, 6)
    else:
        sb, i = 192 * (k // 256), k % 256
        q = ((codes[:, sb + i // 2].int() >> (4 * (i % 2)).int()) & 15) \
            + 16 * ((codes[:, sb + 128 + i // 4].int() >> (2 * (i % 4)).int()) & 3)
    q = torch.where(q >= 32, q - 64, q)
    sc = gm[:, k // 16].double()
    return q * torch.where(sc >= 128, sc - 256, sc) * st[:, k // 256]


def _rows64(s):
    step = max(1, (1 << 25) // s["K"])
    return [(n, min(s["N"], n + step)) for n in range(0, s["N"], step)]


def _act64(g, act):
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    if act == "gelu_tanh":
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        p = torch.sigmoid(2 * z)  # (1 + tanh z) / 2
        return g * p, p + g * 2 * p * torch.sigmoid(-2 * z) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
    p = torch.special.ndtr(g)
    return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    M, N, K, op = case["M"], case["N"], case["K"], case["op"]
    if op == "checkpoint":
        v = s["x"].double()
        v = torch.cat((v, torch.zeros((M, -K % 16), dtype=torch.float64, device="cuda")), 1).reshape(M, -1, 16)
        top = v.abs().amax(-1)
        e = torch.frexp(top)[1] - 7  # the largest magnitude in [64, 128) steps of 2^e
        e = e + (torch.ldexp(top, -e) >= 127.5)
        e = torch.clamp(e, min=-126)[..., None]
        v = torch.ldexp(torch.round(torch.ldexp(v, -e)), e)
        return {"restored": v.reshape(M, -1)[:, :K]}
    F = N // 2
    if op in ("gated", "step"):
        x = s["x"].double()
        gu = torch.empty((M, N), dtype=torch.float64, device="cuda")
        for n0, n1 in _rows64(s):
            gu[:, n0:n1] = x @ _weights64(s, n0, n1).T
        out = {"h": _act64(gu[:, :F], case["act"])[0] * gu[:, F:]}
        if op == "step":
            # (g, u) pass through a rounding to 8 bits: a sum in 32 bits and one in 64 may fall on two sides of
            # a border, so the gradients have no one value here ("backward" starts from given codes and has)
            out["dx"] = None
            if case["dgu"]:
                out["dgu"] = None
        return out
    if op == "dx":
        d = s["dy"].double()
    else:
        codes, e = s["saved"]
        v = torch.ldexp(codes.double().reshape(2 * M, -1, 16), e.int()[..., None] - 127).reshape(M, 2, -1)[..., :F]
        a, da = _act64(v[:, 0], case["act"])
        dh = s["dh"].double()
        d = torch.cat((dh * v[:, 1] * da, dh * a), 1)
    dx = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    for n0, n1 in _rows64(s):
        dx += d[:, n0:n1] @ _weights64(s, n0, n1)
    out = {"dx": dx}
    if case["dgu"]:
        out["dgu"] = d
    return out
