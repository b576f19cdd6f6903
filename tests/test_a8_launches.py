"""Which kernels the 8-bit activation calls launch, recorded without a GPU: a
refused call launches nothing, and the SwiGLU with 8-bit results takes two
launches and scratch memory only where its one launch would leave compute
units without work."""

import re

import pytest

import bit_weight_only_q4g64_amd as q4
from tests.a8_shapes import BF16_KERNELS, PAIRS, PRODUCTS
from tests.launch_record import available, record

pytestmark = pytest.mark.skipif(not available, reason="needs the ROCm compilers")


def test_a_refused_call_launches_nothing():
    """Sizes around the most lanes a launch may have (2^32), where one of two launches could fit and the other not."""
    calls = [("quant", 2**24, 2048), ("quant", 2**24, 2**20), ("norm", 2**24, 2048), ("norm", 2**24, 16384)]
    for m in range(4, 25):
        for n in range(6, 31):
            for k in (64, 2048, 16384, 20480, 65536, 2**20):
                if n + k.bit_length() <= 40:
                    calls += [("swiglu", 2**m, 2**n, k), ("product", 2**m, 2**n, k, "bf16"), ("pair", 2**m, 2**n, k, "f32")]
    refused = 0
    for call, r in zip(calls, record(calls)):
        assert r.status in (q4.Q4_OK, q4.Q4_EINVAL, q4.Q4_EUNSUPPORTED), call
        assert (len(r.launches) > 0) == (r.status == q4.Q4_OK), (call, r)
        assert all(x.workgroups * x.lanes < 2**32 for x in r.launches), (call, r)
        refused += r.status != q4.Q4_OK
    assert refused > 100


def test_scratch_memory_stays_small():
    """M x N float32 values of scratch memory for few workgroups only, however long K is (768 of 64 x 128 at most)."""
    need = q4.a8_swiglu_work_bytes
    for M, N, K in ((8192, 8192, 20480), (4096, 8192, 28672), (8192, 8192, 65536), (2**18, 2**17, 16384), (2048, 28672, 2**20)):
        assert need(M, N, K) == 0, (M, N, K)
    sizes = [(2**m + d, 2**n, k) for m in range(4, 21) for d in (0, 1) for n in range(6, 20) for k in (64, 1024, 8192, 16384, 20480, 2**16, 2**20)]
    assert max(need(*s) for s in sizes) <= 768 * 64 * 128 * 4
    # few workgroups still take the two launches
    for M, N, K in ((16, 1024, 8192), (4, 8192, 2048), (5474, 320, 10944), (1226, 1600, 10368),
                    (12, 67648, 11008), (11008, 320, 10368)):
        assert need(M, N, K) == M * N * 4, (M, N, K)


def test_launches_agree_with_the_scratch_memory():
    calls = [("swiglu", M, N, K) for M in (1, 16, 17, 300, 5474, 8192) for N in (64, 320, 1600, 8192) for K in (64, 2048, 10368, 20480)]
    for call, r in zip(calls, record(calls)):
        assert r.status == q4.Q4_OK and len(r.launches) == (2 if r.work_bytes else 1), (call, r)
        assert r.work_bytes == q4.a8_swiglu_work_bytes(*call[1:]), call


def tile_of(kernel):
    """(rows, columns, the fewest groups of K that turn the loads' ring twice, places the ring can end at) of a product
    kernel by its template arguments, and whether its weights are loaded past the caches."""
    kind, args, flags = re.fullmatch(r"q4::a8_(tile|direct)_kernel<q4::\w+<(.*)>, (.*)>", kernel).groups()
    a = [{"true": 1, "false": 0}.get(v, v) for v in args.split(", ")]
    if kind == "tile":
        exact, pair, wm, wn, mt, ns, ahead, _ = map(int, a)
        return wm * mt * 32, wn * ns * 32 // (1 + pair), 2 * (ahead + 2) + 1, ahead if exact else ahead + 1, flags.endswith("true")
    _, mt, nt, _, nw, kw, ahead = map(int, a)
    return mt * 16, nw * nt * 16, kw * (ahead + 1) + 1, 1, False  # kw waves share the groups


def test_shapes_take_every_kernel_through_its_pipeline():
    """Of every kernel that the sizes of a wide grid launch, tests/a8_shapes.py holds sizes with row and column ends inside
    its tile, half a group at the end of K, and K long enough for two turns of the ring, ending at each of its places."""
    grid = [(M, N, K) for M in (1, 17, 33, 64, 100, 128, 200, 300, 520, 1000, 2000, 4000, 8192) for N in (64, 256, 1024, 2048, 4096, 16384, 65536)
            for K in (64, 256, 1024, 2048, 8192)]
    forms = [("product", "f32"), ("product", "bf16"), ("pair", "f32"), ("pair", "bf16"), ("swiglu", "")]

    def kernels(sizes, ops):
        calls = [(op, *s, out) for s in sizes for op, out in forms if op in ops]
        return [(c[1:4], x.kernel) for c, r in zip(calls, record(calls)) for x in r.launches if "quant" not in x.kernel]

    wanted = {k for _, k in kernels(grid, ("product", "pair", "swiglu"))}
    assert len(wanted) >= 30
    seen = kernels([s[:3] for s in PRODUCTS], ("product",)) + kernels([s[:3] for s in PAIRS], ("pair", "swiglu"))
    for kernel in sorted(wanted):
        rows, cols, groups, places, past_caches = tile_of(kernel)
        ends = {(-(-K // 128) % places, K % 128 != 0) for (M, N, K), k in seen
                if k == kernel and -(-K // 128) >= groups and M % rows and (cols <= 64 or N % cols)}
        assert any(half for _, half in ends), kernel
        if not past_caches:  # the same kernel but for the kind of load
            assert {e for e, _ in ends} == set(range(places)), (kernel, ends)
            assert "direct" in kernel or any(k == kernel and M > 2 * rows and N > 2 * cols for (M, N, K), k in seen), kernel


def test_sizes_of_every_bfloat16_kernel():
    def kernels(sizes):
        return {x.kernel for r in record([("product", *s, "bf16") for s in sizes]) for x in r.launches}

    grid = [(M, N, 1088) for M in (1, 17, 50, 100, 200, 400, 700, 1500, 3000, 8000) for N in (64, 256, 448, 1024, 1344, 2048, 4096, 8192)]
    assert kernels(grid) == kernels(BF16_KERNELS) and len(kernels(BF16_KERNELS)) == len(BF16_KERNELS)
