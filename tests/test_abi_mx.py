"""Host-side refusals of the microscaled entry points: every call returns before
any CUDA call, so none needs a GPU."""
import ctypes
import re

import pytest

from doubly_stochastic_projection_b200 import build

P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
FAKE = 1 << 20  # never dereferenced
OK, NULL, ALIGN, SIZE, ARG = 0, 1, 2, 3, 4

# name: (pointers, required, sizes that are right, does a format follow, iteration count)
MIX = {
    "mhc_residual_mix_fwd_ckpt": (9, range(9), True, False),
    "mhc_proj_mix_fwd_ckpt": (10, range(10), True, True),
    "mhc_residual_mix_bwd_ckpt": (12, [0, 1, 2, 3, 4, 5, 6, 7, 10], True, False),
    "mhc_mix_post_bwd_ckpt": (6, range(6), True, False),
    "mhc_mix_premap_bwd_ckpt": (10, [0, 1, 2, 3, 4, 5, 6, 8], True, False),
    "mhc_premap_fwd_mx4": (4, range(4), False, False),
}


@pytest.fixture(scope="module")
def L():
    return ctypes.CDLL(build.build())


def entry(L, name, pointers, ints):
    f = getattr(L, name)
    f.argtypes = [P] * pointers + ints + [P]
    return f


@pytest.mark.parametrize("name", sorted(MIX))
def test_mix_entry_points(L, name):
    n, required, fmt, iters = MIX[name]
    f = entry(L, name, n, [I64, I64] + [I32] * (fmt + iters))

    def call(ptrs=None, T=4, C=64, it=0, form=0):
        return f(*(ptrs or [FAKE] * n), T, C, *([it] if iters else []), *([form] if fmt else []), None)

    assert call(C=12) == SIZE and call(C=0) == SIZE and call(T=-1) == SIZE and call(T=1 << 36, C=1 << 24) == SIZE
    assert call([None] * n, T=0) == OK
    if fmt:
        assert call(form=2) == ARG and call(form=3) == ARG and call(form=-1) == ARG  # 8-bit formats only
    if iters:
        assert call(it=1001) == ARG and call(it=-1) == ARG
    for k in range(n):
        if k in required:
            assert call([None if i == k else FAKE for i in range(n)]) == NULL, k
        assert call([FAKE + 8 if i == k else FAKE for i in range(n)]) == ALIGN, k


@pytest.mark.parametrize("name", ["mhc_mx_pack", "mhc_mx_unpack"])
def test_pack_entry_points(L, name):
    f = entry(L, name, 3, [I64, I64, I32])
    a = [FAKE] * 3
    assert f(*a, -1, 64, 0, None) == SIZE and f(*a, 4, 60, 0, None) == SIZE and f(*a, 4, 0, 0, None) == SIZE
    assert f(*a, 1 << 38, 64, 0, None) == SIZE
    assert f(*a, 4, 64, 3, None) == ARG and f(*a, 4, 64, -1, None) == ARG
    assert f(None, None, None, 0, 64, 2, None) == OK
    for k in range(3):
        assert f(*[None if i == k else FAKE for i in range(3)], 4, 64, 1, None) == NULL
        assert f(*[FAKE + 4 if i == k else FAKE for i in range(3)], 4, 64, 1, None) == ALIGN


@pytest.mark.parametrize("name,n", [("mhc_mx4_linear", 5), ("mhc_mx4_linear_mix", 8)])
def test_product_entry_points(L, name, n):
    f = entry(L, name, n, [I64, I64, I64])
    a = [FAKE] * n
    for T, N, K in [(-1, 64, 64), (4, 0, 64), (4, 12, 64), (4, 64, 0), (4, 64, 40), (4, 64, 16), ((1 << 31) - 512, 64, 64),
                    (1 << 30, 1 << 24, 64), (1 << 30, 64, 1 << 24), (4, 1 << 25, 64), (4, 64, 1 << 25)]:
        assert f(*a, T, N, K, None) == SIZE, (T, N, K)
    assert f(*[None] * n, 0, 64, 64, None) == OK
    for k in range(n):
        assert f(*[None if i == k else FAKE for i in range(n)], 4, 64, 64, None) == NULL
        assert f(*[FAKE + 2 if i == k else FAKE for i in range(n)], 4, 64, 64, None) == ALIGN


def test_scale_pitch_is_the_header_s():
    from doubly_stochastic_projection_b200 import api

    text = open(build.INCLUDE + "/mhc_birkhoff.h").read()
    assert re.search(r"#define MHC_MX_SCALE_PITCH\(C\) \(4 \* \(\(\(int64_t\)\(C\) \+ 127\) / 128\)\)", text)
    assert [api.mx_scale_pitch(C) for C in (8, 32, 128, 136, 4096)] == [4, 4, 4, 8, 128]


def test_waits_that_run_out_have_a_status_of_their_own(L):
    L.mhc_status_string.restype = ctypes.c_char_p
    L.mhc_status_string.argtypes = [ctypes.c_int]
    assert b"MHC_ERR_WAIT" in L.mhc_status_string(6)
    f = entry(L, "mhc_mx4_linear_diag", 5, [I64, I64, I64, I64, I32])
    a = [FAKE] * 5
    assert f(*a, 4, 12, 64, 1000, 0, None) == SIZE
    for wait_ns, idle in [(0, 0), (-1, 0), (2_000_000_001, 0), (1000, -1), (1000, 16)]:
        assert f(*a, 4, 64, 64, wait_ns, idle, None) == ARG, (wait_ns, idle)
    assert f(*[None] * 5, 0, 64, 64, 1000, 1, None) == OK
    for k in range(5):
        assert f(*[None if i == k else FAKE for i in range(5)], 4, 64, 64, 1000, 1, None) == NULL
        assert f(*[FAKE + 2 if i == k else FAKE for i in range(5)], 4, 64, 64, 1000, 1, None) == ALIGN


def test_roles_that_do_not_exist_are_refused():
    from doubly_stochastic_projection_b200 import api

    with pytest.raises(ValueError):
        api.mx4_linear_diag(None, None, idle=("epilogue",))
