"""Cases and plain forms of the microscaled operators: 8-bit checkpoints of the
residual streams with the backward that reads them, and the 4-bit read map,
product and product-with-mix of serving.

A microscaled row holds blocks of 32 channels with one power-of-two scale each
(a byte, exponent + 127; scale rows are padded with zero bytes to a multiple of
four).  Formats: "int8" (m / 64, |m| <= 127), "e4m3", "e2m1" (two codes a byte,
the even channel in the low half).  The scale is the smallest power of two at
which the block's largest magnitude does not pass the format's largest value.
"""
import torch

own = False

EMAX = {"int8": 0, "e4m3": 8, "e2m1": 2}
TOP = {"int8": 127 / 64, "e4m3": 1.75, "e2m1": 1.5}  # mantissa of the largest value
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a checkpoint written and restored for a recomputed block: streams of 2048 tokens
        {"name": "pack_int8", "op": "pack", "fmt": "int8", "T": 2048, "C": 7168},
        # the same with a ragged last block, and few rows
        {"name": "pack_e4m3_ragged", "op": "pack", "fmt": "e4m3", "T": 777, "C": 1048},
        # training: mix forward with checkpoint and the backward from it, the usual size
        {"name": "train_int8", "op": "train", "fmt": "int8", "T": 16384, "C": 4096},
        # training at an odd width and token count
        {"name": "train_e4m3_odd", "op": "train", "fmt": "e4m3", "T": 1000, "C": 3080},
        # training of a short sequence: latency counts
        {"name": "train_short", "op": "train", "fmt": "int8", "T": 33, "C": 1040},
        # the split backward of a whole layer, at the largest size
        {"name": "layer_bwd_int8_large", "op": "layer_bwd", "fmt": "int8", "T": 65536, "C": 7168},
        # the split backward of a mid-sized batch
        {"name": "layer_bwd_e4m3", "op": "layer_bwd", "fmt": "e4m3", "T": 3000, "C": 4096},
        # decoding one token: read map, 4-bit codes, the layer's first product
        {"name": "read4_one", "op": "read4", "T": 1, "C": 7168, "N": 8192},
        # a small batch, ragged output width
        {"name": "read4_odd", "op": "read4", "T": 200, "C": 4096, "N": 4104},
        # a long prompt
        {"name": "read4_prompt", "op": "read4", "T": 8192, "C": 4096, "N": 8192},
        # decoding one token: the layer's last product with the mix
        {"name": "write4_one", "op": "write4", "T": 1, "K": 8192, "C": 4096},
        # a long prompt
        {"name": "write4_prompt", "op": "write4", "T": 16384, "K": 8192, "C": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["pack", "train", "layer_bwd", "read4", "write4"])
    if op in ("pack", "train", "layer_bwd"):
        C = 8 * _log(rng, 16, 960)
        T = _log(rng, 1, min(65536, (1 << 26) // C))
        return {"op": op, "fmt": rng.choice(["int8", "e4m3"]), "T": T, "C": C}
    T = _log(rng, 1, 8192)
    if op == "read4":
        return {"op": op, "T": T, "C": 32 * _log(rng, 16, 224), "N": 8 * _log(rng, 64, 1024)}
    return {"op": op, "T": T, "K": 32 * _log(rng, 16, 256), "C": 8 * _log(rng, 64, 896)}


def work(case):
    T, C = case["T"], case["C"]
    q8, q4 = 1 + 1 / 32, 0.5 + 1 / 32
    if case["op"] == "pack":
        return {"bytes": 4 * T * C * (2 + q8 + q8 + 2), "flops": 4 * T * C * 4}
    if case["op"] == "train":
        fwd = T * (10 * C + 8 * C + 5 * C * q8 + 80)
        bwd = T * (8 * C + 5 * C * q8 + 10 * C + 160)
        return {"bytes": fwd + bwd, "flops": T * C * (40 + 80)}
    if case["op"] == "layer_bwd":
        return {"bytes": T * (8 * C + q8 * C + 2 * C + 8 * C + 4 * q8 * C + 2 * C + 8 * C + 180), "flops": T * C * 96}
    if case["op"] == "read4":
        N = case["N"]
        return {"bytes": 8 * T * C + N * C * q4 + 2 * T * N, "flops": 2 * T * N * C + 8 * T * C}
    K = case["K"]
    return {"bytes": 2 * T * K + C * K * q4 + 16 * T * C, "flops": 2 * T * C * K + 40 * T * C}


# ---------------------------------------------------------------- the format, plainly

def _pitch(C):
    return 4 * ((C + 127) // 128)


def _blocks(x):
    C = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -C % 32))
    return x.view(*x.shape[:-1], -1, 32)


def _scale_byte(amax, fmt):
    """The scale's byte of each block from its largest magnitude (float32)."""
    over = (1 << 23) - 1 - round((TOP[fmt] - 1) * (1 << 23))  # carries into the exponent above the top mantissa
    e = ((amax.view(torch.int32) + over) >> 23) - EMAX[fmt]
    return torch.where(torch.isfinite(amax), e.clamp(0, 254), 255)


def _scale(byte):
    """2^(byte - 127) as float32, exactly (byte 0 is a subnormal number)."""
    bits = torch.where(byte > 0, byte << 23, 1 << 22)
    return torch.where(byte < 255, bits.view(torch.float32), float("nan"))


def _round(q, fmt):
    if fmt == "int8":
        return (q * 64).round().clamp(-127, 127) / 64
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).float()
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((a / step).round() * step, q)


def _values(x, fmt):
    """What the codes of x stand for, as float32, of x's shape."""
    b = _blocks(x)
    s = _scale(_scale_byte(b.abs().amax(-1), fmt))[..., None]
    return (_round(b / s, fmt) * s).flatten(-2)[..., :x.shape[-1]]


def _pack(x, fmt):
    """Codes and scales of x in the layout that a user's program holds."""
    C = x.shape[-1]
    b = _blocks(x)
    byte = _scale_byte(b.abs().amax(-1), fmt)
    q = _round(b / _scale(byte)[..., None], fmt).flatten(-2)[..., :C]
    if fmt == "int8":
        codes = (q * 64).to(torch.int8).view(torch.uint8)
    elif fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        a = q.abs()
        c = (a * 2).long() - (a > 2).long() - (a > 3).long() * 1 - (a > 4).long() * 3
        c = (c + 8 * torch.signbit(q)).to(torch.uint8)
        codes = c[..., 0::2] | (c[..., 1::2] << 4)
    scales = torch.nn.functional.pad(byte.to(torch.uint8), (0, _pitch(C) - byte.shape[-1]))
    return codes.contiguous(), scales.contiguous()


def _unpack(codes, scales, fmt, dtype=torch.float32):
    """The values that codes and scales stand for."""
    if fmt == "int8":
        q = codes.view(torch.int8).float() / 64
    elif fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        q = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)[c]
    C = q.shape[-1]
    s = _scale(scales.int()).repeat_interleave(32, -1)[..., :C]
    return q.to(dtype) * s.to(dtype)


# ---------------------------------------------------------------- inputs

def _streams(g, *shape):
    """bf16 activations: normal, with a few channels that are much larger."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    gain = torch.ones(shape[-1], device="cuda", dtype=torch.bfloat16)
    gain[torch.randint(shape[-1], (max(1, shape[-1] // 200),), generator=g, device="cuda")] = 16
    return x * gain


def _maps(g, T):
    p = torch.randn((T, 4, 4), generator=g, device="cuda").exp()
    for _ in range(20):
        p = p / p.sum(-1, keepdim=True)
        p = p / p.sum(-2, keepdim=True)
    return p.contiguous(), torch.rand((T, 4), generator=g, device="cuda") * 2


def _weight(g, n, k):
    return _pack(torch.randn((n, k), generator=g, device="cuda", dtype=torch.bfloat16) * k ** -0.5, "e2m1")


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    T, C, op = case["T"], case["C"], case["op"]
    s = {"op": op, "fmt": case.get("fmt"), "T": T, "C": C}
    if op == "pack":
        s["X"] = _streams(g, T, 4, C)
        return s
    H, h = _maps(g, T)
    if op == "train":
        s |= {"X": _streams(g, T, 4, C), "F": _streams(g, T, C), "H": H, "h": h}
        s["dY"] = torch.randn((T, 4, C), generator=g, device="cuda", dtype=torch.bfloat16)
    elif op == "layer_bwd":
        # the checkpoints that the forward left
        s["Xq"] = _pack(_streams(g, T, 4, C), case["fmt"])
        s["Fq"] = _pack(_streams(g, T, C), case["fmt"])
        s |= {"H": H, "h": h, "h_pre": torch.randn((T, 4), generator=g, device="cuda")}
        s["dY"] = torch.randn((T, 4, C), generator=g, device="cuda", dtype=torch.bfloat16)
        s["dx_in"] = torch.randn((T, C), generator=g, device="cuda", dtype=torch.bfloat16)
    elif op == "read4":
        s |= {"X": _streams(g, T, 4, C), "h_pre": torch.randn((T, 4), generator=g, device="cuda")}
        s["W"] = _weight(g, case["N"], C)
    else:
        s |= {"A": _streams(g, T, case["K"]), "X": _streams(g, T, 4, C), "H": H, "h": h}
        s["W"] = _weight(g, C, case["K"])
    return s


# ---------------------------------------------------------------- one pass

def _run_own(s):
    from doubly_stochastic_projection_b200 import api

    op, fmt = s["op"], s["fmt"]
    if op == "pack":
        return api.mx_unpack(api.mx_pack(s["X"], fmt))
    if op == "train":
        Y, Xq, Fq = api.residual_mix_fwd_ckpt(s["X"], s["H"], s["h"], s["F"], fmt)
        d = api.residual_mix_bwd_ckpt(Xq, s["H"], s["h"], Fq, s["dY"])
        return {"Y": Y, "dX": d["dX"], "dF": d["dF"], "dH": d["dH_res"], "dh": d["dh_post"]}
    if op == "layer_bwd":
        dF, dh = api.mix_post_bwd_ckpt(s["dY"], api.MxTensor(*s["Fq"], fmt), s["h"])
        d = api.mix_premap_bwd_ckpt(api.MxTensor(*s["Xq"], fmt), s["H"], s["h_pre"], s["dY"], s["dx_in"],
                                    need_dH=True, need_dlogits=False)
        return {"dX": d["dX"], "dF": dF, "dH": d["dH_res"], "dh": dh, "dh_pre": d["dh_pre"]}
    w = api.MxTensor(*s["W"], "e2m1")
    if op == "read4":
        return api.mx4_linear(api.premap_fwd_mx4(s["X"], s["h_pre"]), w)
    return api.mx4_linear_mix(api.mx_pack(s["A"], "e2m1"), w, s["X"], s["H"], s["h"])


def _run_plain(s):
    op, fmt, bf = s["op"], s["fmt"], torch.bfloat16
    if op == "pack":
        return _values(s["X"], fmt).to(bf)
    if op == "train":
        H, h, dY = s["H"], s["h"], s["dY"].float()
        Y = (H @ s["X"].float() + h[..., None] * s["F"].float()[:, None]).to(bf)
        X, F = _values(s["X"], fmt), _values(s["F"], fmt)
        return {"Y": Y, "dX": (H.mT @ dY).to(bf), "dF": (h[:, None] @ dY)[:, 0].to(bf),
                "dH": dY @ X.mT, "dh": (dY @ F[..., None])[..., 0]}
    if op == "layer_bwd":
        H, h, dY, dx = s["H"], s["h"], s["dY"].float(), s["dx_in"].float()
        X, F = _unpack(*s["Xq"], fmt), _unpack(*s["Fq"], fmt)
        w = torch.sigmoid(s["h_pre"])
        e = (-s["h_pre"].abs()).exp()
        return {"dX": (H.mT @ dY + w[..., None] * dx[:, None]).to(bf), "dF": (h[:, None] @ dY)[:, 0].to(bf),
                "dH": dY @ X.mT, "dh": (dY @ F[..., None])[..., 0],
                "dh_pre": e / (1 + e) ** 2 * (X @ dx[..., None])[..., 0]}
    W = _unpack(*s["W"], "e2m1")
    if op == "read4":
        x_in = (torch.sigmoid(s["h_pre"])[:, None] @ s["X"].float())[:, 0]
        return (_values(x_in, "e2m1") @ W.T).to(bf)
    F = _values(s["A"], "e2m1") @ W.T
    return (s["H"] @ s["X"].float() + s["h"][..., None] * F[:, None]).to(bf)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- in 64 bits

def _grid64(x, fmt):
    """x rounded to the format's values, from the definition, in float64."""
    x = x.double()
    C = x.shape[-1]
    x = torch.cat((x, x.new_zeros(*x.shape[:-1], -C % 32)), -1).unflatten(-1, (-1, 32))
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # amax = 2m * 2^(e - 1), 1 <= 2m < 2
    e = (e - 1 - EMAX[fmt] + (2 * m > TOP[fmt])).clamp(-127, 127).double()
    q = x * torch.exp2(-e)
    low, bits = {"int8": (0, 6), "e4m3": (-6, 3), "e2m1": (0, 1)}[fmt]
    if fmt == "int8":
        step = torch.full_like(q, 2.0 ** -6)
    else:
        step = torch.exp2((torch.frexp(q)[1] - 1).clamp(min=low).double() - bits)
    top = TOP[fmt] * 2 ** EMAX[fmt]
    q = ((q / step).round() * step).clamp(-top, top)
    return (q * torch.exp2(e)).flatten(-2)[..., :C]


def _decode64(codes, scales, fmt):
    if fmt == "int8":
        q = codes.view(torch.int8).double() * 2.0 ** -6
    elif fmt == "e4m3":
        c = codes.long()
        e, m = (c >> 3) & 15, (c & 7).double()
        q = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9) * (1 - 2 * (c >> 7)).double()
    else:
        c = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.long, device=codes.device)
        c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
        e, m = (c >> 1) & 3, (c & 1).double()
        q = torch.where(e > 0, (2 + m) * torch.exp2(e.double() - 2), m * 0.5) * (1 - 2 * (c >> 3)).double()
    s = torch.exp2(scales.double() - 127)
    return q * s[..., torch.arange(q.shape[-1], device=q.device) // 32]


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt, T = s["op"], s["fmt"], s["T"]
    rows = max(1, (1 << 27) // (16 * s["C"]))  # tokens at a time: 64-bit streams are large
    parts = []
    for a in range(0, T, rows):
        cut = slice(a, a + rows)
        if op == "pack":
            parts.append({"": _grid64(s["X"][cut], fmt)})
            continue
        if op == "read4":
            w = 1 / (1 + (-s["h_pre"][cut].double()).exp())
            x = _grid64((w[..., None] * s["X"][cut].double()).sum(1), "e2m1")
            parts.append({"": x @ _decode64(*s["W"], "e2m1").T})
            continue
        H, h = s["H"][cut].double(), s["h"][cut].double()
        if op == "write4":
            F = _grid64(s["A"][cut], "e2m1") @ _decode64(*s["W"], "e2m1").T
            parts.append({"": torch.einsum("tij,tjc->tic", H, s["X"][cut].double()) + h[:, :, None] * F[:, None, :]})
            continue
        dY = s["dY"][cut].double()
        out = {"dX": torch.einsum("tij,tic->tjc", H, dY), "dF": torch.einsum("ti,tic->tc", h, dY)}
        if op == "train":
            X, F = _grid64(s["X"][cut], fmt), _grid64(s["F"][cut], fmt)
            out["Y"] = torch.einsum("tij,tjc->tic", H, s["X"][cut].double()) + h[:, :, None] * s["F"][cut].double()[:, None, :]
        else:
            X = _decode64(s["Xq"][0][cut], s["Xq"][1][cut], fmt)
            F = _decode64(s["Fq"][0][cut], s["Fq"][1][cut], fmt)
            dx, w = s["dx_in"][cut].double(), 1 / (1 + (-s["h_pre"][cut].double()).exp())
            out["dX"] += w[:, :, None] * dx[:, None, :]
            out["dh_pre"] = w * (1 - w) * torch.einsum("tc,tjc->tj", dx, X)
        out["dH"] = torch.einsum("tic,tjc->tij", dY, X)
        out["dh"] = torch.einsum("tic,tc->ti", dY, F)
        # the streams' gradients are kept in 32 bits where they are many: 2^-24 is far below their bf16 rounding
        parts.append({k: v.float() if k in ("Y", "dX", "dF") else v for k, v in out.items()})
    whole = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    return whole[""] if "" in whole else whole
