"""GPU tests of microscaled storage, the 8-bit checkpoints of the residual
streams with the backward that reads them, and the 4-bit read map and products,
against the fp64 oracles (oracle/mx.py, oracle.c).

Codes and scales are compared bit for bit: the scale is a power of two, so the
element's rounding is the only one.  Tolerances count roundings: half a step
of bf16 is 2^-8 of the value, an fp32 sum of n terms is off by at most
n 2^-24 times the sum of the terms' magnitudes (to first order; n counts the
roundings on the longest path, and is rounded up below).
"""
import numpy as np
import pytest
import torch

from doubly_stochastic_projection_b200 import api, inputs
from oracle import mx
from _gpu_util import GRAD_REL_TOL, bf16_bits, dev, per_matrix_rel_err, row_normalised, to_gpu, to_np64

pytestmark = pytest.mark.gpu

FORMATS = ("int8", "e4m3", "e2m1")
CKPT = ("int8", "e4m3")
BF16 = 2.0 ** -8
FP32 = 2.0 ** -24


def np_u8(t):
    return t.cpu().numpy()


def streams(shape, seed, outliers=True):
    """bf16 rows whose blocks differ in scale."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 7, shape[:-1] + (1,)))
    if outliers:
        x[..., rng.integers(shape[-1])] *= 40
    return torch.from_numpy(x.astype(np.float32)).to(dev()).bfloat16()


def assert_codes(got, x64, fmt):
    codes, scales = mx.pack(x64, fmt)
    np.testing.assert_array_equal(np_u8(got.scales), scales)
    np.testing.assert_array_equal(np_u8(got.codes), codes)


# ------------------------------------------------------------------ storage

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R,C", [(1, 8), (3, 24), (5, 32), (130, 40), (7, 128), (33, 136), (9, 1048), (2, 4104),
                                 (1000, 256), (1, 32768)])
def test_pack_and_unpack(fmt, R, C):
    x = streams((R, C), R + C)
    q = api.mx_pack(x, fmt)
    assert q.shape == (R, C) and q.scales.shape == (R, api.mx_scale_pitch(C))
    assert_codes(q, to_np64(x), fmt)
    y = api.mx_unpack(q)
    np.testing.assert_array_equal(to_np64(y), mx.unpack(np_u8(q.codes), np_u8(q.scales), fmt))


def as_bf16(v64):
    """float64 values rounded to bf16.  Codes of bf16 inputs stand for bf16 numbers,
    but the e4m3 and e2m1 elements next to 2^128 round up to it, which bf16 has
    as infinity; codes that no pack makes may also fall under its smallest number."""
    with np.errstate(over="ignore", invalid="ignore"):
        return torch.from_numpy(v64).float().bfloat16().double().numpy()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("C", [64, 72])
def test_rows_on_sixteen_byte_boundaries_only(fmt, C):
    # the alignment that is asked for is 16 bytes: rows that start between two
    # 32-byte boundaries, in and out
    flat = streams((1, 8 + 20 * C), 7)[0]
    x = flat[8:].view(20, C)
    assert x.data_ptr() % 32 == 16
    q = api.mx_pack(x, fmt)
    assert_codes(q, to_np64(x), fmt)
    out = torch.full((16 + 20 * C,), 7.0, dtype=torch.bfloat16, device=dev())
    y = api.mx_unpack(q, out=out[8:8 + 20 * C].view(20, C))
    assert torch.equal(y, api.mx_unpack(q))
    assert (out[:8] == 7).all() and (out[8 + 20 * C:] == 7).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_restores(fmt):
    codes = np.arange(256, dtype=np.uint8)[None].repeat(256, 0)  # row r: every code at scale r
    C = 512 if fmt == "e2m1" else 256
    scales = np.zeros((256, api.mx_scale_pitch(C)), np.uint8)
    scales[:, :C // 32] = np.arange(256, dtype=np.uint8)[:, None]
    y = api.mx_unpack(api.MxTensor(to_gpu(codes), to_gpu(scales), fmt))
    np.testing.assert_array_equal(to_np64(y), as_bf16(mx.unpack(codes, scales, fmt)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_values(fmt):
    x = torch.ones((6, 200), dtype=torch.bfloat16, device=dev())
    x[0, 5], x[0, 70], x[0, 199] = float("inf"), float("nan"), -float("inf")
    x[1] = 0
    x[2] = -0.0
    x[3] = torch.finfo(torch.bfloat16).max
    x[4] = 2.0 ** -133
    x[4, 50] = 2.0 ** -126
    x[4, 100] = 127 * 2.0 ** -133
    x[5, :32] = torch.finfo(torch.bfloat16).min
    q = api.mx_pack(x, fmt)
    assert_codes(q, to_np64(x), fmt)
    y = api.mx_unpack(q)
    np.testing.assert_array_equal(to_np64(y), as_bf16(mx.unpack(np_u8(q.codes), np_u8(q.scales), fmt)))
    assert torch.isnan(y[0, :32]).all() and torch.isnan(y[0, 64:96]).all() and torch.isnan(y[0, 192:]).all()
    assert (y[0, 32:64] == 1).all() and (y[0, 96:192] == 1).all()


def test_all_bf16_values_alone_in_a_block():
    bits = np.arange(65536, dtype=np.uint16)
    x = torch.zeros((65536, 32), dtype=torch.bfloat16, device=dev())
    x[:, 7] = torch.from_numpy(bits.view(np.int16)).to(dev()).view(torch.bfloat16)
    for fmt in FORMATS:
        assert_codes(api.mx_pack(x, fmt), to_np64(x), fmt)


# -------------------------------------------- forward and backward, training

def _case(T, C, seed=3):
    m = inputs.mix_workload("mix_T16384_C4096", device=dev(), T=T, C=C)
    X, F = streams((T, 4, C), seed), streams((T, C), seed + 1)
    H = api.birkhoff_fwd(to_gpu(m["logits"]), "newton")
    return X, F, m["dY"], H, to_gpu(m["h_post"]), to_gpu(m["logits"])


def _sum_bound(C, absolute):
    # a thread adds its vectors of 8 one after the other, then 5 + 4 levels across the CTA
    n = 8 * -(-C // 1024) + 9
    return 2 * n * FP32 * absolute


def _check_reductions(out, Xr, Fr, dY, names=("dH_res", "dh_post")):
    C = dY.shape[-1]
    if "dH_res" in names:
        ref = np.einsum("tic,tjc->tij", dY, Xr)
        assert (np.abs(to_np64(out["dH_res"]) - ref) <= _sum_bound(C, np.einsum("tic,tjc->tij", abs(dY), abs(Xr)))).all()
    if "dh_post" in names:
        ref = np.einsum("tic,tc->ti", dY, Fr)
        assert (np.abs(to_np64(out["dh_post"]) - ref) <= _sum_bound(C, np.einsum("tic,tc->ti", abs(dY), abs(Fr)))).all()


@pytest.mark.parametrize("fmt", CKPT)
@pytest.mark.parametrize("T,C", [(1, 8), (2, 1024), (3, 1048), (17, 4096), (5, 7168), (300, 1032), (3000, 264)])
def test_mix_with_checkpoint(orc, fmt, T, C):
    X, F, dY, H, h, logits = _case(T, C)
    Y, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F, fmt)
    assert torch.equal(Y, api.residual_mix_fwd(X, H, h, F))
    assert_codes(Xq, to_np64(X), fmt)
    assert_codes(Fq, to_np64(F), fmt)
    Y2, H2, Xq2, Fq2 = api.proj_mix_fwd_ckpt(logits, h, X, F, fmt)
    Y3, H3 = api.proj_mix_fwd(logits, h, X, F)
    assert (H2 - H3).abs().max().item() <= 2e-6
    # Y moves with H by at most |dH| |X|_1, and by a bf16 step
    tol = 2e-6 * X.float().abs().sum(1, keepdim=True) + 2 * BF16 * Y3.float().abs()
    assert ((Y2.float() - Y3.float()).abs() <= tol).all()
    for a, b in zip(Xq + Fq, Xq2 + Fq2):
        assert a == b if isinstance(a, str) else torch.equal(a, b)

    out = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY, need_dlogits=True)
    plain = api.residual_mix_bwd(X, H, h, F, dY)
    assert torch.equal(out["dX"], plain["dX"]) and torch.equal(out["dF"], plain["dF"])
    Xr, Fr = api.mx_unpack(Xq), api.mx_unpack(Fq)
    _check_reductions(out, to_np64(Xr), to_np64(Fr), to_np64(dY))
    # the chained projection backward, from the oracle's dH at the restored streams
    dH = np.einsum("tic,tjc->tij", to_np64(dY), to_np64(Xr))
    ref = orc.implicit_bwd(row_normalised(to_np64(H)), dH)
    rel, _ = per_matrix_rel_err(to_np64(out["dlogits"]), ref)
    assert rel.max() <= GRAD_REL_TOL, rel.max()
    dX, dl, dh, dF = api.proj_mix_bwd_ckpt(H, h, Xq, Fq, dY)
    assert torch.equal(dX, out["dX"]) and torch.equal(dF, out["dF"])
    assert torch.equal(dl, out["dlogits"]) and torch.equal(dh, out["dh_post"])
    # outputs that are not asked for are not written, the others do not change
    few = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY, need_dH=False, need_dh_post=False)
    assert few["dH_res"] is None and few["dh_post"] is None and few["dlogits"] is None
    assert torch.equal(few["dX"], out["dX"]) and torch.equal(few["dF"], out["dF"])


@pytest.mark.parametrize("fmt", CKPT)
@pytest.mark.parametrize("T,C", [(1, 8), (2, 1032), (33, 4096), (700, 1048)])
def test_split_backward_from_checkpoint(orc, fmt, T, C):
    X, F, dY, H, h, _ = _case(T, C, 11)
    Xq, Fq = api.mx_pack(X, fmt), api.mx_pack(F, fmt)
    Xr, Fr = api.mx_unpack(Xq), api.mx_unpack(Fq)
    h_pre = to_gpu((np.random.default_rng(5).standard_normal((T, 4)) * 3).astype(np.float32))
    dx_in = inputs.bf16_normal((T, C), 77, dev())
    dF, dh = api.mix_post_bwd_ckpt(dY, Fq, h)
    dF0, dh0 = api.mix_post_bwd(dY, Fr, h)
    assert torch.equal(dF, dF0)
    _check_reductions({"dh_post": dh}, None, to_np64(Fr), to_np64(dY), ("dh_post",))
    out = api.mix_premap_bwd_ckpt(Xq, H, h_pre, dY, dx_in, need_dH=True, need_dlogits=True)
    ref = api.mix_premap_bwd(Xr, H, h_pre, dY, dx_in, need_dH=True, need_dlogits=True)
    assert torch.equal(out["dX"], ref["dX"])
    _check_reductions(out, to_np64(Xr), None, to_np64(dY), ("dH_res",))
    s = 1 / (1 + np.exp(-to_np64(h_pre)))
    g = s * (1 - s)
    dot = np.einsum("tc,tjc->tj", to_np64(dx_in), to_np64(Xr))
    mag = np.einsum("tc,tjc->tj", abs(to_np64(dx_in)), abs(to_np64(Xr)))
    # the sigmoid's derivative carries a few fp32 roundings of its own
    assert (np.abs(to_np64(out["dh_pre"]) - g * dot) <= _sum_bound(C, g * mag) + 16 * FP32 * np.abs(g * dot)).all()
    dH = np.einsum("tic,tjc->tij", to_np64(dY), to_np64(Xr))
    rel, _ = per_matrix_rel_err(to_np64(out["dlogits"]), orc.implicit_bwd(row_normalised(to_np64(H)), dH))
    assert rel.max() <= GRAD_REL_TOL, rel.max()
    few = api.mix_premap_bwd_ckpt(Xq, H, h_pre, dY, dx_in, need_dH=False, need_dlogits=False)
    assert few["dH_res"] is None and few["dlogits"] is None and torch.equal(few["dh_pre"], out["dh_pre"])


def test_gradient_from_checkpoint_against_differences():
    # L = <dY, Y(H, h)> is linear in H and h, so a difference of the forward at
    # the restored streams is the derivative, up to the bf16 rounding of Y
    T, C, fmt = 4, 512, "int8"
    X, F, dY, H, h, _ = _case(T, C, 21)
    _, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F, fmt)
    out = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY)
    Xr, Fr = api.mx_unpack(Xq), api.mx_unpack(Fq)
    d64 = to_np64(dY)
    for i in range(4):
        for j in range(4):
            E = torch.zeros_like(H)
            E[:, i, j] = 1.0
            Y = to_np64(api.residual_mix_fwd(Xr, E, torch.zeros_like(h), Fr))
            diff = np.einsum("tic,tic->t", d64, Y)
            tol = BF16 * np.einsum("tic,tic->t", abs(d64), abs(Y)) + _sum_bound(C, np.einsum("tc,tc->t", abs(d64[:, i]), abs(to_np64(Xr)[:, j])))
            assert (np.abs(to_np64(out["dH_res"])[:, i, j] - diff) <= tol).all()
        e = torch.zeros_like(h)
        e[:, i] = 1.0
        Y = to_np64(api.residual_mix_fwd(Xr, torch.zeros_like(H), e, Fr))
        diff = np.einsum("tic,tic->t", d64, Y)
        tol = BF16 * np.einsum("tic,tic->t", abs(d64), abs(Y)) + _sum_bound(C, np.einsum("tc,tc->t", abs(d64[:, i]), abs(to_np64(Fr))))
        assert (np.abs(to_np64(out["dh_post"])[:, i] - diff) <= tol).all()


def test_non_finite_tokens_stay_their_own():
    T, C = 5, 136
    X, F, dY, H, h, _ = _case(T, C, 31)
    X[2, 1, 40] = float("inf")
    F[3, 0] = float("nan")
    _, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F)
    out = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY)
    dH, dh = out["dH_res"], out["dh_post"]
    assert torch.isnan(dH[2, :, 1]).all() and torch.isfinite(dH[2][:, [0, 2, 3]]).all()
    assert torch.isnan(dh[3]).all()
    assert torch.isfinite(dH[[0, 1, 3, 4]]).all() and torch.isfinite(dh[[0, 1, 2, 4]]).all()
    assert torch.isfinite(out["dX"]).all() and torch.isfinite(out["dF"]).all()


@pytest.mark.parametrize("fmt", CKPT)
def test_autograd_keeps_checkpoints_only(fmt):
    T, C = 200, 1048
    X, F, dY, H, h, logits = _case(T, C, 41)
    X, F, H, h, logits = (t.clone().requires_grad_(True) for t in (X, F, H, h, logits))
    Y = api.ResidualMixCkpt.apply(X, H, h, F, fmt)
    saved = [t for t in Y.grad_fn.saved_tensors]
    assert all(t.dtype != torch.bfloat16 for t in saved)
    Y.backward(dY)
    with torch.no_grad():
        _, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F, fmt)
        ref = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY)
    assert torch.equal(X.grad, ref["dX"]) and torch.equal(F.grad, ref["dF"])
    assert torch.equal(H.grad, ref["dH_res"]) and torch.equal(h.grad, ref["dh_post"])
    X.grad = F.grad = h.grad = None
    api.ProjectedMixCkpt.apply(logits, h, X, F, fmt).backward(dY)
    with torch.no_grad():
        _, H2, Xq, Fq = api.proj_mix_fwd_ckpt(logits, h, X, F, fmt)
        dX, dl, dh, dF = api.proj_mix_bwd_ckpt(H2, h, Xq, Fq, dY)
    assert torch.equal(X.grad, dX) and torch.equal(F.grad, dF)
    assert torch.equal(logits.grad, dl) and torch.equal(h.grad, dh)


def test_layers_with_checkpoints_run_together():
    # a stack of layers, trained with checkpoints: the gradients are those of the
    # same stack whose backward is given the restored streams
    T, C, L = 64, 520, 3
    X, _, dY, _, _, _ = _case(T, C, 51)
    rng = np.random.default_rng(52)
    logits = [to_gpu(rng.standard_normal((T, 4, 4)).astype(np.float32)).requires_grad_(True) for _ in range(L)]
    h = [to_gpu(rng.uniform(0, 2, (T, 4)).astype(np.float32)).requires_grad_(True) for _ in range(L)]
    x = X.clone().requires_grad_(True)
    ins, hid = [], x
    for lg, hp in zip(logits, h):
        F = hid.mean(1)  # a layer of its own: plain torch
        ins.append((hid.detach(), F.detach()))
        hid = api.ProjectedMixCkpt.apply(lg, hp, hid, F, "int8")
    hid.backward(dY)
    g = dY
    for lg, hp, (xi, Fi) in reversed(list(zip(logits, h, ins))):
        with torch.no_grad():
            _, H, Xq, Fq = api.proj_mix_fwd_ckpt(lg, hp, xi, Fi, "int8")
            dX, dl, dh, dF = api.proj_mix_bwd_ckpt(H, hp, Xq, Fq, g)
        assert torch.equal(lg.grad, dl) and torch.equal(hp.grad, dh)
        z = xi.clone().requires_grad_(True)
        z.mean(1).backward(dF)
        g = dX + z.grad
    assert torch.equal(x.grad, g)


# ------------------------------------------------------------------ 4 bits

@pytest.mark.parametrize("T,C", [(1, 8), (1, 7168), (3, 1048), (40, 4096), (1000, 136)])
def test_read_map_to_four_bits(T, C):
    X = streams((T, 4, C), T)
    h_pre = to_gpu((np.random.default_rng(T).standard_normal((T, 4)) * 2).astype(np.float32))
    q = api.premap_fwd_mx4(X, h_pre)
    s = 1 / (1 + np.exp(-to_np64(h_pre)))
    x64 = to_np64(X)
    ref = np.einsum("tj,tjc->tc", s, x64)
    # fp32: the weights' roundings and four products
    off = 12 * FP32 * np.einsum("tj,tjc->tc", s, abs(x64))
    S = np_u8(q.scales)[:, :-(-C // 32)]
    pad = ((0, 0), (0, -C % 32))
    lo, hi = (mx.scale_bytes(np.abs(np.pad(ref, pad)) + d * np.pad(off, pad), "e2m1") for d in (-1, 1))
    assert (S >= lo).all() and (S <= hi).all()  # equal but next to a border
    assert (np.mean(lo != hi) < 1e-3) and (np_u8(q.scales)[:, -(-C // 32):] == 0).all()
    # each element is the nearest at the scale that was taken, up to fp32's error at a tie
    y = mx.unpack(np_u8(q.codes), np_u8(q.scales), "e2m1")
    sc = np.repeat(2.0 ** (S.astype(float) - 127), 32, -1)[:, :C]
    e, _ = mx.elements(ref / sc, "e2m1")
    best = np.abs(np.abs(ref) / sc - mx.TABLE["e2m1"][e]) * sc
    assert (np.abs(y - ref) <= best + 2 * off).all()


def _operands(T, N, K, seed):
    a, w = streams((T, K), seed), streams((N, K), seed + 1, outliers=False)
    return api.mx_pack(a, "e2m1"), api.mx_pack(w, "e2m1")


def _values(q):
    return mx.unpack(np_u8(q.codes), np_u8(q.scales), "e2m1")


def _product_bound(K, mag):
    # a block's products are exact; the blocks' sums are added in fp32, an
    # addition being off by at most a step (2^-23) of the running magnitude
    return (K // 32 + 8) * 2 * FP32 * mag


# the forms of the product: one tile shared along K in tiles of 16 and of 64
# tokens, and (from 149 tiles of 64 tokens on) persistent tiles of 192
PRODUCTS = [(1, 8, 32), (1, 136, 512), (2, 264, 96), (7, 1032, 1056), (16, 512, 4096), (17, 520, 2048), (33, 128, 256),
            (64, 4104, 320), (65, 384, 288), (129, 256, 1024), (200, 1000, 544), (257, 136, 4128), (1030, 200, 352),
            (1, 19000, 512), (16, 18952, 96), (200, 8200, 1056), (513, 2200, 1024), (2500, 520, 544), (700, 4104, 4128),
            (9600, 136, 256), (385, 3080, 1536)]


@pytest.mark.parametrize("T,N,K", PRODUCTS)
def test_product(T, N, K):
    a, w = _operands(T, N, K, T + N)
    out = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device=dev())
    got = api.mx4_linear(a, w, out=out[:T])
    ref, mag = _values(a) @ _values(w).T, np.abs(_values(a)) @ np.abs(_values(w)).T
    assert (np.abs(to_np64(got) - ref) <= BF16 * np.abs(ref) + 2 * _product_bound(K, mag)).all()
    assert (out[T:] == 7).all()  # rows behind the last token are left alone
    api.wait_status()
    assert torch.equal(got, api.mx4_linear(a, w))  # and the sums' order is fixed


@pytest.mark.parametrize("T,C,K", PRODUCTS)
def test_product_with_mix(T, C, K):
    a, w = _operands(T, C, K, T + C)
    X = streams((T, 4, C), T)
    rng = np.random.default_rng(K)
    H = api.birkhoff_fwd(to_gpu(rng.standard_normal((T, 4, 4)).astype(np.float32)), "newton")
    h = to_gpu(rng.uniform(0, 2, (T, 4)).astype(np.float32))
    out = torch.full((T + 1, 4, C), 7.0, dtype=torch.bfloat16, device=dev())
    got = api.mx4_linear_mix(a, w, X, H, h, out=out[:T])
    F, mag = _values(a) @ _values(w).T, np.abs(_values(a)) @ np.abs(_values(w)).T
    ref = np.einsum("tij,tjc->tic", to_np64(H), to_np64(X)) + to_np64(h)[:, :, None] * F[:, None]
    terms = np.einsum("tij,tjc->tic", to_np64(H), abs(to_np64(X))) + to_np64(h)[:, :, None] * abs(F)[:, None]
    tol = BF16 * np.abs(ref) + 2 * to_np64(h)[:, :, None] * _product_bound(K, mag)[:, None] + 8 * FP32 * terms
    assert (np.abs(to_np64(got) - ref) <= tol).all()
    assert (out[T:] == 7).all()
    assert torch.equal(got, api.mx4_linear_mix(a, w, X, H, h))


@pytest.mark.parametrize("T,N,K", [(3, 264, 2048), (300, 6200, 2048)])
def test_product_of_operands_on_sixteen_byte_boundaries(T, N, K):
    a, w = _operands(T, N, K, 5)

    def moved(t):
        flat = torch.empty(t.numel() + 16, dtype=torch.uint8, device=dev())[16:]
        assert flat.data_ptr() % 32 == 16
        return flat.view(t.shape).copy_(t)

    b, v = (api.MxTensor(moved(q.codes), moved(q.scales), q.fmt) for q in (a, w))
    out = torch.empty(T * N + 8, dtype=torch.bfloat16, device=dev())[8:].view(T, N)
    assert torch.equal(api.mx4_linear(b, v, out=out), api.mx4_linear(a, w))


def test_bytes_behind_the_last_scale_do_not_count():
    # scale rows are padded to four bytes; what a caller left in the padding is not read
    a, w = _operands(5, 40, 160, 6)
    ref = api.mx4_linear(a, w)
    for q in (a, w):
        q.scales[:, 5:] = 255
    assert torch.equal(api.mx4_linear(a, w), ref)


def test_product_of_special_blocks():
    # NaN blocks reach their own token or channel only; zero rows give zeros
    T, N, K = 40, 72, 256
    x, wt = streams((T, K), 1), streams((N, K), 2, outliers=False)
    x[3, 40] = float("nan")
    x[5] = 0
    wt[9, 200] = float("inf")
    wt[11] = 0
    out = api.mx4_linear(api.mx_pack(x, "e2m1"), api.mx_pack(wt, "e2m1"))
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[3], want[:, 9] = True, True
    assert torch.equal(nan, want)
    keep = [n for n in range(N) if n != 9]
    assert (out[5][keep] == 0).all() and (out[[t for t in range(T) if t != 3], 11] == 0).all()


def test_serving_layer_runs_together():
    # read map -> codes -> first product -> activation -> codes -> last product with the mix
    for T in (1, 70):
        C, N = 1024, 2048
        X = streams((T, 4, C), T, outliers=False)
        rng = np.random.default_rng(9)
        h_pre = to_gpu(rng.standard_normal((T, 4)).astype(np.float32))
        H = api.birkhoff_fwd(to_gpu(rng.standard_normal((T, 4, 4)).astype(np.float32)), "newton")
        h = to_gpu(rng.uniform(0, 2, (T, 4)).astype(np.float32))
        w1 = api.mx_pack(streams((N, C), 5, outliers=False), "e2m1")
        w2 = api.mx_pack(streams((C, N), 6, outliers=False), "e2m1")
        x4 = api.premap_fwd_mx4(X, h_pre)
        u = torch.relu(api.mx4_linear(x4, w1))
        u4 = api.mx_pack(u, "e2m1")
        Y = api.mx4_linear_mix(u4, w2, X, H, h)
        assert_codes(u4, to_np64(u), "e2m1")
        F = _values(u4) @ _values(w2).T
        ref = np.einsum("tij,tjc->tic", to_np64(H), to_np64(X)) + to_np64(h)[:, :, None] * F[:, None]
        scale = np.abs(_values(u4)) @ np.abs(_values(w2)).T
        tol = BF16 * np.abs(ref) + 4 * _product_bound(N, scale)[:, None] + 8 * FP32 * np.abs(to_np64(X)).sum(1)[:, None]
        assert (np.abs(to_np64(Y) - ref) <= tol).all()


def _product_us(T, N, K, calls=20):
    """Least time of a product on the device, calls back to back."""
    a, w = _operands(T, N, K, 85)
    out = api.mx4_linear(a, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            api.mx4_linear(a, w, out=out)
    best = float("inf")
    for _ in range(20):
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        graph.replay()
        t1.record()
        t1.synchronize()
        best = min(best, t0.elapsed_time(t1) / calls * 1e3)
    del graph
    return best


@pytest.mark.parametrize("T", (1, 16, 64))
def test_clusters_that_share_a_tile_run_in_one_wave(T):
    # 32 tiles fit the GPU in clusters of 4; 16 tiles do not in clusters of 8, of
    # which the GPCs hold fewer than SMs / 8.  Half the work in one wave takes no
    # longer than all of it, in two waves nearly twice as long: the bound is between
    assert _product_us(T, 2048, 4096) <= 1.4 * _product_us(T, 4096, 4096)


@pytest.mark.parametrize("role", sorted(api.MX4_ROLES))
@pytest.mark.parametrize("T,N,K", [(3, 264, 2080), (3, 264, 32768), (60, 264, 32768), (1500, 2056, 4128)])
def test_a_wait_that_runs_out(T, N, K, role):
    # a role that does nothing: the others wait for it in vain, each for a
    # millisecond, and return.  In all three forms, with K tiles for each stage and
    # more, and (the first) with so few that some role has no wait left
    a, w = _operands(T, N, K, 81)
    ref = api.mx4_linear(a, w)
    api.wait_status()
    out = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device=dev())
    api.mx4_linear_diag(a, w, wait_ns=1_000_000, idle=(role,), out=out[:T])
    with pytest.raises(api.MhcError) as e:
        api.wait_status()
    assert e.value.status == 6
    api.wait_status()  # said once
    assert torch.isnan(out[:T]).all() and (out[T:] == 7).all()
    # the next product has its shared and tensor memory whole, on every SM
    assert torch.equal(api.mx4_linear(a, w), ref)
    assert torch.equal(api.mx4_linear_diag(a, w), ref)
    api.wait_status()


# ---------------------------------------------------- streams, graphs, refusals

def test_side_streams_and_graph_replay():
    T, C, N = 136, 1024, 520  # X[:, 0] also serves as weights: T is a multiple of 8
    X, F, dY, H, h, _ = _case(T, C, 61)
    w = api.mx_pack(streams((C, N * 4), 62, outliers=False), "e2m1")
    act = streams((T, N * 4), 63)

    def run():
        Y, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F)
        d = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, dY)
        Z = api.mx4_linear_mix(api.mx_pack(act, "e2m1"), w, X, H, h)
        V = api.mx4_linear(api.premap_fwd_mx4(X, h), api.mx_pack(X[:, 0].contiguous(), "e2m1"))
        return [Y, d["dX"], d["dF"], d["dH_res"], d["dh_post"], Z, V, api.mx_unpack(Xq)]

    ref = run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(dev()), torch.cuda.Stream(dev())
    for _ in range(3):
        got = []
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(run())
        s1.synchronize()
        s2.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for k in range(3):
        for t in out:
            t.zero_()
        if k == 2:  # new inputs in the captured buffers
            X.copy_(streams((T, 4, C), 64))
            ref = run()
            torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    del g


@pytest.mark.parametrize("T", (1, 16, 200, 2500))
def test_product_follows_its_operands(T):
    # one operand's buffers, written anew for each product while the last may still run
    N = K = 1024
    w = api.mx_pack(streams((N, K), 71, outliers=False), "e2m1")
    xs = [streams((T, K), 72 + i, outliers=False) for i in range(4)]
    h_pre = to_gpu(np.random.default_rng(73).standard_normal((T, 4)).astype(np.float32))
    ref = []
    for x in xs:
        a = api.mx_pack(x, "e2m1")
        torch.cuda.synchronize()
        u = api.mx4_linear(a, w)
        torch.cuda.synchronize()
        b = api.premap_fwd_mx4(torch.stack([u, x, u, x], 1), h_pre)
        torch.cuda.synchronize()
        ref.append(api.mx4_linear(b, w))
        torch.cuda.synchronize()
    a = api.mx_pack(xs[0], "e2m1")
    X = torch.empty((T, 4, K), dtype=torch.bfloat16, device=dev())
    u = torch.empty((T, N), dtype=torch.bfloat16, device=dev())

    def chain():
        got = []
        for x in xs:
            api.mx_pack(x, "e2m1", out=a)
            api.mx4_linear(a, w, out=u)
            for j in range(4):
                X[:, j].copy_(x if j & 1 else u)
            got.append(api.mx4_linear(api.premap_fwd_mx4(X, h_pre), w))
        return got

    for _ in range(20):
        assert all(torch.equal(g, r) for g, r in zip(chain(), ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(out, ref))
    del graph


@pytest.mark.parametrize("K", (544, 1536, 2048))  # scale rows of 20, 48 and 64 bytes: loads of 4, 16 and 32
@pytest.mark.parametrize("T,N", [(1, 1024), (40, 1024), (700, 2048)])
def test_product_follows_its_scales_and_maps(T, N, K):
    # as above, at every width of the scales' loads, and with maps and weights that
    # the kernels just before it wrote
    xs = [streams((T, K), 90 + i, outliers=False) for i in range(3)]
    ws = [streams((N, K), 93 + i, outliers=False) for i in range(3)]
    rng = np.random.default_rng(96)
    lg = [to_gpu(rng.standard_normal((T, 4, 4)).astype(np.float32)) for _ in xs]
    h = to_gpu(rng.uniform(0, 2, (T, 4)).astype(np.float32))
    X = streams((T, 4, N), 97)
    a, w, H = api.mx_pack(xs[0], "e2m1"), api.mx_pack(ws[0], "e2m1"), api.birkhoff_fwd(lg[0])

    def chain(wait):
        got = []
        for x, wt, l in zip(xs, ws, lg):
            steps = (lambda: api.mx_pack(wt, "e2m1", out=w), lambda: api.mx_pack(x, "e2m1", out=a),
                     lambda: got.append(api.mx4_linear(a, w)), lambda: api.mx_pack(x, "e2m1", out=a),
                     lambda: api.birkhoff_fwd(l, out=H), lambda: got.append(api.mx4_linear_mix(a, w, X, H, h)))
            for f in steps:
                f()
                wait()
        return got

    ref = chain(torch.cuda.synchronize)
    for _ in range(10):
        assert all(torch.equal(g, r) for g, r in zip(chain(lambda: None), ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(lambda: None)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(out, ref))
    del graph


def test_empty_batches():
    d = dev()
    for fmt in FORMATS:
        q = api.mx_pack(torch.empty((0, 64), dtype=torch.bfloat16, device=d), fmt)
        assert q.shape == (0, 64) and api.mx_unpack(q).shape == (0, 64)
    X, F = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=d), torch.empty((0, 64), dtype=torch.bfloat16, device=d)
    H, h = torch.empty((0, 4, 4), device=d), torch.empty((0, 4), device=d)
    Y, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F)
    assert api.residual_mix_bwd_ckpt(Xq, H, h, Fq, Y)["dX"].shape == (0, 4, 64)
    a = api.premap_fwd_mx4(X, h)
    w = api.mx_pack(torch.ones((64, 64), dtype=torch.bfloat16, device=d), "e2m1")
    assert api.mx4_linear(a, w).shape == (0, 64)
    assert api.mx4_linear_mix(a, w, X, H, h).shape == (0, 4, 64)


def test_binding_refusals():
    d = dev()
    x = torch.ones((4, 64), dtype=torch.bfloat16, device=d)
    X, H, h = torch.ones((4, 4, 64), dtype=torch.bfloat16, device=d), torch.ones((4, 4, 4), device=d), torch.ones((4, 4), device=d)
    q8, q4 = api.mx_pack(x, "int8"), api.mx_pack(x, "e2m1")
    with pytest.raises(ValueError):
        api.mx_pack(x, "int4")
    with pytest.raises(TypeError):
        api.mx_pack(x.float(), "int8")
    with pytest.raises(ValueError):
        api.mx_pack(x.cpu(), "int8")
    with pytest.raises(ValueError):
        api.mx_pack(x.t(), "int8")
    with pytest.raises(api.MhcError) as e:
        api.mx_pack(torch.ones((4, 12), dtype=torch.bfloat16, device=d), "int8")
    assert e.value.status == 3
    with pytest.raises(ValueError):
        api.mx_pack(x, "int8", out=q4)
    with pytest.raises(ValueError):
        api.residual_mix_fwd_ckpt(X, H, h, x, "e2m1")
    with pytest.raises(TypeError):
        api.residual_mix_bwd_ckpt(X, H, h, q8, X)
    with pytest.raises(ValueError):  # two formats
        api.residual_mix_bwd_ckpt(api.mx_pack(X, "e4m3"), H, h, q8, X)
    with pytest.raises(ValueError):  # scales of another width
        api.mx_unpack(api.MxTensor(q8.codes, q8.scales[:, :2].contiguous(), "int8"))
    with pytest.raises(ValueError):
        api.mx4_linear(q8, q8)
    with pytest.raises(ValueError):  # inner sizes differ
        api.mx4_linear(q4, api.mx_pack(torch.ones((8, 96), dtype=torch.bfloat16, device=d), "e2m1"))
    with pytest.raises(api.MhcError) as e:  # K not a multiple of the block
        y = api.mx_pack(torch.ones((8, 40), dtype=torch.bfloat16, device=d), "e2m1")
        api.mx4_linear(y, y)
    assert e.value.status == 3
    with pytest.raises(api.MhcError) as e:  # N not a multiple of 8
        api.mx4_linear(q4, api.mx_pack(torch.ones((4, 64), dtype=torch.bfloat16, device=d), "e2m1"))
    assert e.value.status == 3


# --------------------------------------------------- offsets past 32 bits

def _tail_equals(whole, part, n):
    return all(torch.equal(w[-n:], p) for w, p in zip(whole, part))


def test_offsets_past_32_bits():
    # streams of 4.9e9 elements: the last tokens come out as they do alone
    T, C, n = 300_000, 4096, 3
    d = dev()
    g = torch.Generator(d).manual_seed(1)
    X = torch.randn((T, 4, C), generator=g, device=d, dtype=torch.bfloat16)
    F = torch.randn((T, C), generator=g, device=d, dtype=torch.bfloat16)
    H, h = torch.rand((T, 4, 4), generator=g, device=d), torch.rand((T, 4), generator=g, device=d)
    cut = [t[-n:].contiguous() for t in (X, H, h, F)]
    Y, Xq, Fq = api.residual_mix_fwd_ckpt(X, H, h, F)
    Y1, Xq1, Fq1 = api.residual_mix_fwd_ckpt(*cut)
    assert _tail_equals((Y, *Xq[:2], *Fq[:2]), (Y1, *Xq1[:2], *Fq1[:2]), n)
    q = api.mx_pack(X, "int8")
    assert torch.equal(q.codes, Xq.codes) and torch.equal(q.scales, Xq.scales)
    del q
    torch.cuda.empty_cache()
    assert torch.equal(api.mx_unpack(Xq)[-n:], api.mx_unpack(Xq1))
    out = api.residual_mix_bwd_ckpt(Xq, H, h, Fq, Y, need_dlogits=True)
    one = api.residual_mix_bwd_ckpt(Xq1, cut[1], cut[2], Fq1, Y1, need_dlogits=True)
    assert all(torch.equal(out[k][-n:], one[k]) for k in out)
    del out, Y
    torch.cuda.empty_cache()
    dF, dh = api.mix_post_bwd_ckpt(X, Fq, h)
    assert _tail_equals((dF, dh), api.mix_post_bwd_ckpt(cut[0], Fq1, cut[2]), n)
    out = api.mix_premap_bwd_ckpt(Xq, H, h, X, F)
    one = api.mix_premap_bwd_ckpt(Xq1, cut[1], cut[2], cut[0], cut[3])
    assert torch.equal(out["dX"][-n:], one["dX"]) and torch.equal(out["dh_pre"][-n:], one["dh_pre"])
    del out, dF, Xq, Fq
    torch.cuda.empty_cache()
    a = api.premap_fwd_mx4(X, h)
    assert _tail_equals(a[:2], api.premap_fwd_mx4(cut[0], cut[2])[:2], n)
    # the product's forms sum in different orders: compared within two roundings of its terms
    a = api.mx_pack(torch.randn((T, 64), generator=g, device=d, dtype=torch.bfloat16), "e2m1")
    w = api.mx_pack(torch.randn((C * 4, 64), generator=g, device=d, dtype=torch.bfloat16), "e2m1")
    part = api.MxTensor(a.codes[-n:].clone(), a.scales[-n:].clone(), "e2m1")
    big, small = api.mx4_linear(a, w)[-n:].float(), api.mx4_linear(part, w).float()
    assert ((big - small).abs() <= 2 * BF16 * small.abs() + 1e-4).all()
    w = api.MxTensor(w.codes[:C].clone(), w.scales[:C].clone(), "e2m1")
    Z = api.mx4_linear_mix(a, w, X, H, h)[-n:].float()
    Z1 = api.mx4_linear_mix(part, w, cut[0], cut[1], cut[2]).float()
    assert ((Z - Z1).abs() <= 2 * BF16 * Z1.abs() + 1e-4).all()
    api.wait_status()
    del X, F, Z, big, a
    torch.cuda.empty_cache()
