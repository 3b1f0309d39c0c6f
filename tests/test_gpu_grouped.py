"""GPU: products grouped by expert and products with a fused epilogue,
against float64 at group sizes, shapes and epilogues where they can go
wrong."""
import numpy as np
import pytest

from mlp_huffman_coded_b200 import synth
from mlp_huffman_coded_b200 import uw
from oracle import uw_oracle as O

from gpu_util import bf16_f64, device_matrix, empty_bf16, to_dev, to_host_u16
from moe_util import (F32, HALF_ULP, SMALLEST_NORMAL, act_tail, activation_bound, check_slots, epilogue_bound,
                      expert_weights, grouped_ref, swiglu_ref)

pytestmark = pytest.mark.gpu


def experts_of(mats):
    return uw.Experts([device_matrix(m) for m in mats])


def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def random_rows(offsets, x_rows, n, seed):
    return np.random.default_rng(seed).integers(0, x_rows, n).astype(np.int32)


def run_grouped(ex, x, offsets, n_rows, rows=None, fp32=False, **epi):
    import torch
    y = torch.full((n_rows, ex.rows), 777.0, dtype=torch.float32, device="cuda")
    if not fp32:
        y = y.to(torch.bfloat16)
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, n_rows))
    epi = {k: (to_dev(v) if isinstance(v, np.ndarray) else v) for k, v in epi.items()}
    uw.gemm_grouped(ex, to_dev(x), to_dev(offsets), y, ws, rows=None if rows is None else to_dev(rows), **epi)
    ws.check("gemm_grouped")
    assert int(ws.t[256:256 + 65536].sum()) == 0  # the counters are back at zero
    return y.double().cpu().numpy()


# group sizes: none, one row, ragged, one group with all rows, tile borders
COUNTS = [[0, 0, 0, 1], [1, 0, 5, 17], [16, 15, 0, 33], [0, 70, 0, 0], [64, 128, 1, 3], [300, 0, 2, 257]]


@pytest.mark.parametrize("shape", [(256, 512), (200, 192), (1, 64), (129, 1088)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_against_float64(shape, counts):
    rows, cols = shape
    E = len(counts)
    mats = expert_weights(E, rows, cols, 500)
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(max(n // 2, 3), cols, 501)
    r = random_rows(off, x.shape[0], n, 502)
    ex = experts_of(mats)
    for fp32 in (False, True):
        got = run_grouped(ex, x, off, n, rows=r, fp32=fp32)
        ok, worst = check_slots(got, grouped_ref(mats, x, r, off, bf16=not fp32))
        assert ok, (fp32, worst)


def test_grouped_one_token_per_expert_many_experts():
    E, rows, cols = 70, 128, 128
    mats = expert_weights(E, rows, cols, 520)
    counts = [1 if e % 3 else 0 for e in range(E)]
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(n, cols, 521)
    got = run_grouped(experts_of(mats), x, off, n)
    ok, worst = check_slots(got, grouped_ref(mats, x, np.arange(n), off))
    assert ok, worst


def test_slots_outside_the_groups_stay_as_they_were():
    mats = expert_weights(3, 256, 256, 530)
    off = offsets_of([5, 0, 9], first=4)
    n = 40
    x = synth.activations(n, 256, 531)
    got = run_grouped(experts_of(mats), x, off, n)
    untouched = float(O.bf16_to_f64(synth.f32_to_bf16_bits(np.array([777.0], np.float32)))[0])
    assert np.all(got[:4] == untouched) and np.all(got[18:] == untouched)
    ok, worst = check_slots(got, grouped_ref(mats, x, np.arange(n), off))
    assert ok, worst


def test_no_group_has_a_slot():
    mats = expert_weights(2, 256, 256, 535)
    x = synth.activations(9, 256, 536)
    got = run_grouped(experts_of(mats), x, np.array([3, 3, 3], np.int32), 9)
    assert len(set(got.ravel())) == 1  # all as they were


@pytest.mark.parametrize("act", sorted(uw.ACTIVATIONS))
@pytest.mark.parametrize("fp32", [False, True])
def test_grouped_epilogue(act, fp32):
    E, rows, cols = 4, 330, 320
    mats = expert_weights(E, rows, cols, 540)
    off = offsets_of([3, 40, 0, 18])
    n = int(off[-1])
    x = synth.activations(n, cols, 541)
    bias = synth.activations(E, rows, 542)
    res = synth.activations(n, rows, 543)
    ex = experts_of(mats)
    for b, q in ((bias, res), (bias, None), (None, res)):
        got = run_grouped(ex, x, off, n, fp32=fp32, bias=b, activation=act, residual=q)
        ok, worst = check_slots(got, grouped_ref(mats, x, np.arange(n), off, b, act, q, bf16=not fp32))
        assert ok, (b is None, q is None, worst)


@pytest.mark.parametrize("shape", [(256, 512), (130, 64), (1088, 576)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped_swiglu_against_float64(shape, counts):
    rows, cols = shape
    E = len(counts)
    gs, us = expert_weights(E, rows, cols, 550), expert_weights(E, rows, cols, 560)
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(max(n // 2, 3), cols, 551)
    r = random_rows(off, x.shape[0], n, 552)
    eg, eu = experts_of(gs), experts_of(us)
    h = empty_bf16(n, rows)
    ws = uw.Workspace(uw.grouped_workspace_bytes(eg, n, swiglu=True))
    uw.gemm_grouped_swiglu(eg, eu, to_dev(x), to_dev(off), h, ws, rows=to_dev(r))
    ws.check("swiglu")
    ok, worst = check_slots(bf16_f64(to_host_u16(h)), swiglu_ref(gs, us, x, r, off))
    assert ok, worst


@pytest.mark.parametrize("rate", [0.0, 2e-2, 0.5])
def test_many_verbatim_rows_and_mixed_palettes(rate):
    """Tiles with more verbatim rows than are staged on chip (all of them at
    the highest rate), and one expert whose palette spans both halves of the
    exponent range beside experts whose palettes do not."""
    mats = expert_weights(3, 256, 512, 570, rate=rate, scale=300.0)
    wide = np.random.default_rng(571).choice([0.01, 0.02, 1.5, 3.0], size=(256, 512)).astype(np.float32)
    mats[1] = synth.f32_to_bf16_bits(wide * np.random.default_rng(572).choice([-1, 1], size=(256, 512)).astype(np.float32))
    off = offsets_of([20, 9, 31])
    x = synth.activations(60, 512, 573)
    got = run_grouped(experts_of(mats), x, off, 60)
    ok, worst = check_slots(got, grouped_ref(mats, x, np.arange(60), off))
    assert ok, worst


@pytest.mark.parametrize("batch", [1, 16, 17, 49, 63, 65, 100, 256, 257, 600])
@pytest.mark.parametrize("shape", [(256, 512), (1000, 4096)])
def test_epilogue_against_float64(batch, shape):
    rows, cols = shape
    w = synth.weight_matrix(rows, cols, 0.02, 1e-3, 200.0, 580)
    dm = device_matrix(w)
    x = synth.activations(batch, cols, 581)
    bias = synth.activations(1, rows, 582)
    res = synth.activations(batch, rows, 583)
    y = empty_bf16(batch, rows)
    ws = uw.Workspace(uw.epilogue_workspace_bytes(dm, batch))
    uw.gemm_epilogue(dm, to_dev(x), y, ws, bias=to_dev(bias[0]), activation="silu", residual=to_dev(res))
    ws.check()
    ok, worst = check_slots(bf16_f64(to_host_u16(y)),
                            grouped_ref([w], x, np.arange(batch), [0, batch], bias, "silu", res))
    assert ok, worst
    # in place on the residual
    r = to_dev(res)
    uw.gemm_epilogue(dm, to_dev(x), r, ws, bias=to_dev(bias[0]), activation="silu", residual=r)
    ws.check()
    assert np.array_equal(to_host_u16(r), to_host_u16(y))


# ---------------------- schedules of larger products -------------------------
# Waves of whole tiles, shared tiles, column tiles, row-tile pairs, permuted
# and gathered rows.  The float64 reference runs on the GPU (torch.double).

def f64(bits):
    import torch
    return to_dev(bits).view(torch.bfloat16).double()


def device_experts(mats):
    ws = uw.Workspace(256)
    return uw.Experts([uw.DeviceMatrix.encode_on_device(to_dev(m)).prepare_direct_palette(ws, keep_idx4=False) for m in mats])


def worst_excess(y, mats, x, rows, offsets, K, swiglu_with=None):
    """max(|y - ref| - bound) over all slots (bounds of moe_util, on the GPU)."""
    import torch
    worst = -np.inf
    xd = f64(x)
    for e, w in enumerate(mats):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b <= a:
            continue
        xe = xd[torch.from_numpy(rows[a:b].astype(np.int64)).cuda()]
        wd = f64(w)
        v, d = xe @ wd.T, K * 2.0 ** -23 * (xe.abs() @ wd.abs().T)
        if swiglu_with is not None:
            ud = f64(swiglu_with[e])
            u, du = xe @ ud.T, K * 2.0 ** -23 * (xe.abs() @ ud.abs().T)
            s = v / (1 + torch.exp(-v))
            d = 1.1 * d * u.abs() + s.abs() * du + 1.1 * d * du + 16 * 2.0 ** -24 * (v.abs() + s.abs()) * u.abs()
            v = s * u
        if y.dtype != torch.float32:
            d = d + 2.0 ** -8 * (v.abs() + d)
        worst = max(worst, float(((y[a:b].double() - v).abs() - d).max()) - 1e-30)
    return worst


BIG = [  # rows, cols, group sizes
    (4096, 1024, [50, 200, 0, 131, 64, 7, 90, 33]),   # waves and shared tiles
    (14336, 512, [500, 33]),                          # column tiles, waves
    (2048, 1024, [3] * 64),                           # many small groups
    (1096, 8192, [2900, 2860]),                       # row-tile pairs, the last one half empty
    (4096, 4096, [40, 0, 21]),                        # fewer tiles than CTAs, left whole
    (512, 4096, [1, 2]),                              # and shared out
]


@pytest.mark.parametrize("case", range(len(BIG)))
@pytest.mark.parametrize("scattered", [False, True])
def test_larger_products_against_float64(case, scattered):
    import torch
    rows, cols, counts = BIG[case]
    mats = expert_weights(len(counts), rows, cols, 800 + 100 * case, rate=1e-4)
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(n // 2 + 1 if scattered else n, cols, 801)
    r = random_rows(off, x.shape[0], n, 802) if scattered else np.arange(n)
    ex = device_experts(mats)
    y = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, n))
    xd, rd, offd = to_dev(x), to_dev(r.astype(np.int32)) if scattered else None, to_dev(off)
    uw.gemm_grouped(ex, xd, offd, y, ws, rows=rd)
    ws.check()
    assert worst_excess(y, mats, x, r, off, cols) <= 0
    again = torch.empty_like(y)
    uw.gemm_grouped(ex, xd, offd, again, ws, rows=rd)
    ws.check()
    assert torch.equal(y, again)  # the sums do not depend on timing
    z = torch.empty(n, rows, dtype=torch.float32, device="cuda")
    uw.gemm_grouped(ex, xd, offd, z, ws, rows=rd)
    ws.check()
    assert worst_excess(z, mats, x, r, off, cols) <= 0
    assert torch.equal(z.to(torch.bfloat16), y)


@pytest.mark.parametrize("rows,cols,counts", [(4096, 1024, [50, 200, 0, 131]), (14336, 512, [500, 33]), (1000, 2048, [9, 30, 1])])
def test_larger_swiglu_against_float64(rows, cols, counts):
    import torch
    gs, us = expert_weights(len(counts), rows, cols, 900), expert_weights(len(counts), rows, cols, 920)
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(n // 2 + 1, cols, 901)
    r = random_rows(off, x.shape[0], n, 902)
    eg, eu = device_experts(gs), device_experts(us)
    h = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(eg, n, swiglu=True))
    uw.gemm_grouped_swiglu(eg, eu, to_dev(x), to_dev(off), h, ws, rows=to_dev(r))
    ws.check()
    assert worst_excess(h, gs, x, r, off, cols, swiglu_with=us) <= 0


def test_matrices_prepared_again_leave_the_products_as_they_were():
    """A matrix's new pack gets new memory and the old one's would be handed
    out again: Experts keeps it."""
    import torch
    mats = expert_weights(3, 512, 1024, 935)
    ex = experts_of(mats)
    off = offsets_of([5, 0, 30])
    x = synth.activations(35, 1024, 936)
    want = run_grouped(ex, x, off, 35)
    ws = uw.Workspace(256)
    sizes = [m.pack.numel() for m in ex.matrices]
    for m in ex.matrices:
        m.prepare_direct_palette(ws, keep_idx4=False)
    torch.cuda.synchronize()
    taken = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    assert np.array_equal(run_grouped(ex, x, off, 35), want)
    del taken


def test_six_hundred_experts():
    mats = expert_weights(6, 128, 64, 930)
    dms = [device_matrix(m) for m in mats]
    E = 600
    ex = uw.Experts([dms[e % 6] for e in range(E)])  # the same matrix many times
    counts = [(e * 7) % 4 for e in range(E)]
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(n, 64, 931)
    got = run_grouped(ex, x, off, n)
    ok, worst = check_slots(got, grouped_ref([mats[e % 6] for e in range(E)], x, np.arange(n), off))
    assert ok, worst


def test_more_than_two_to_the_31_output_values():
    import torch
    rows, cols, batch = 32768, 64, 66000
    w = synth.weight_matrix(rows, cols, 0.02, 1e-3, 200.0, 940)
    dm = uw.DeviceMatrix.encode_on_device(to_dev(w)).prepare_direct_palette(uw.Workspace(256), keep_idx4=False)
    x = synth.activations(batch, cols, 941)
    y = torch.empty(batch, rows, dtype=torch.bfloat16, device="cuda")
    ws = uw.Workspace(uw.epilogue_workspace_bytes(dm, batch))
    uw.gemm_epilogue(dm, to_dev(x), y, ws)
    ws.check()
    for a in (0, 32760, 65536, batch - 40):
        part = y[a:a + 40]
        assert worst_excess(part, [w], x[a:a + 40], np.arange(40), [0, 40], cols) <= 0
    del y


def random_matrix(rows, cols, seed):
    """BF16 matrix on the GPU: N(0, 0.02), one weight in 10^4 a hundredfold."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(rows, cols, generator=g, device="cuda") * 0.02
    return torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 1e-4, w * 100, w).to(torch.bfloat16)


@pytest.mark.parametrize("rows", [2104, 2101])  # 17 row tiles; the second: no row of y starts on 16 bytes but the first
@pytest.mark.parametrize("scattered", [False, True])
def test_epilogues_of_row_tile_pairs(rows, scattered):
    """Twice the units from which pairs of row tiles share activations, the
    last pair half empty, groups not multiples of 8.  The plain FP32 product
    against float64; the epilogues against float64 forms of that same product,
    so that only their own rounding is allowed."""
    import torch
    cols, counts = 16384, [1099, 1003, 0, 1195]
    ws_ = [random_matrix(rows, cols, 1000 + e) for e in range(4)]
    load = uw.Workspace(256)
    ex = uw.Experts([uw.DeviceMatrix.encode_on_device(w).prepare_direct_palette(load, keep_idx4=False) for w in ws_])
    off = offsets_of(counts)
    n = int(off[-1])
    x = synth.activations(n, cols, 1010)
    r = np.random.default_rng(1011).permutation(n).astype(np.int32) if scattered else np.arange(n, dtype=np.int32)
    xd, rd, offd = to_dev(x), to_dev(r) if scattered else None, to_dev(off)
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, n))
    z = torch.full((n, rows), 777.0, device="cuda")
    uw.gemm_grouped(ex, xd, offd, z, ws, rows=rd)
    ws.check()
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        for part in range(a, b, 400):  # float64 copies of x stay small
            c = min(part + 400, b)
            xe = f64(x[r[part:c]])
            d = cols * 2.0 ** -23 * (xe.abs() @ ws_[e].double().abs().T)
            assert float(((z[part:c].double() - xe @ ws_[e].double().T).abs() - d).max()) <= 0
    bias = to_dev(synth.activations(4, rows, 1012))
    res = to_dev(synth.activations(n, rows, 1013))
    of_slot = torch.repeat_interleave(torch.arange(4, device="cuda"), torch.tensor(counts, device="cuda"))
    bd, qd = bias.view(torch.bfloat16).double()[of_slot], res.view(torch.bfloat16).double()
    for act, b, q, fp32 in (("gelu", bias, res, True), ("gelu", bias, res, False), ("none", bias, None, True),
                            ("relu", None, res, False), ("none", None, None, False)):
        v = z.double() + (0.0 if b is None else bd)
        ref = {"gelu": lambda: 0.5 * v * torch.special.erfc(-v / 2 ** 0.5), "relu": lambda: v.clamp(min=0), "none": lambda: v}[act]()
        # epilogue_bound with an exact sum: the bias's addition through a slope
        # of at most 1.13, the activation's own error, the residual's addition
        d = 1.13 * F32 * v.abs() + (64 * F32 * (v.abs() + ref.abs()) if act == "gelu" else 0.0)
        ref = ref + (0.0 if q is None else qd)
        d = d + F32 * ref.abs() + F32 * d + 1e-30
        d = d if fp32 else d + HALF_ULP * (ref.abs() + d)
        y = torch.full((n, rows), 777.0, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        uw.gemm_grouped(ex, xd, offd, y, ws, rows=rd, bias=b, activation=act, residual=q)
        ws.check()
        assert float(((y.double() - ref).abs() - d).max()) <= 0, (act, fp32)
        if q is not None and not fp32:  # in place on the residual
            t = q.clone()
            uw.gemm_grouped(ex, xd, offd, t, ws, rows=rd, bias=b, activation=act, residual=t)
            ws.check()
            assert torch.equal(t.view(torch.bfloat16), y)


def test_millions_of_rows_of_a_small_matrix():
    """More rows than the narrow tiles that such a matrix prefers can count."""
    import torch
    rows, cols, n = 200, 128, 2_600_003
    mats = expert_weights(2, rows, cols, 945)
    ups = expert_weights(2, rows, cols, 947)
    ex, eu = experts_of(mats), experts_of(ups)
    x = np.resize(synth.activations(4099, cols, 946), (n, cols))
    xd, off = to_dev(x), offsets_of([700_001, n - 700_001])
    y = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, n, swiglu=True))
    spans = [(0, 300, 0), (700_001 - 260, 700_001, 0), (700_001, 700_300, 1), (2**21 - 100, 2**21 + 100, 1), (n - 300, n, 1)]
    uw.gemm_grouped(ex, xd, to_dev(off), y, ws)
    ws.check()
    for a, b, e in spans:
        assert worst_excess(y[a:b], [mats[e]], x[a:b], np.arange(b - a), [0, b - a], cols) <= 0
    back = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")  # rows of x in falling order
    uw.gemm_grouped_swiglu(ex, eu, xd, to_dev(off), y, ws, rows=back)
    ws.check()
    for a, b, e in spans:
        assert worst_excess(y[a:b], [mats[e]], x[n - b:n - a][::-1].copy(), np.arange(b - a), [0, b - a], cols,
                            swiglu_with=[ups[e]]) <= 0
    uw.gemm_epilogue(ex.matrices[1], xd, y, ws)
    ws.check()
    for a, b, _ in spans:
        assert worst_excess(y[a:b], [mats[1]], x[a:b], np.arange(b - a), [0, b - a], cols) <= 0


# ------------------------------ special values -------------------------------

def test_nan_and_infinite_activations_stay_in_their_slot():
    mats = expert_weights(2, 256, 256, 950)
    off = offsets_of([20, 13])
    x = synth.activations(33, 256, 951)
    clean = run_grouped(experts_of(mats), x, off, 33)
    x[4, 7] = 0x7FC0    # NaN
    x[25, 100] = 0x7F80  # +inf
    got = run_grouped(experts_of(mats), x, off, 33)
    keep = np.ones(33, bool)
    keep[[4, 25]] = False
    assert np.array_equal(got[keep], clean[keep])
    assert np.isnan(got[4]).all() and not np.isfinite(got[25]).any()


def test_weights_of_every_bf16_pattern():
    """Infinities, NaNs, zeros and subnormals among the weights: y is what the
    IEEE sum gives, row by row."""
    w = synth.all_patterns_matrix()  # 1024 x 64
    finite = np.isfinite(O.bf16_to_f64(w)).all(axis=1)
    dm = device_matrix(w)
    x = synth.f32_to_bf16_bits(np.eye(64, dtype=np.float32)[:8])  # picks out columns
    import torch
    y = torch.empty(8, 1024, dtype=torch.float32, device="cuda")
    ws = uw.Workspace(uw.epilogue_workspace_bytes(dm, 8))
    uw.gemm_epilogue(dm, to_dev(x), y, ws)
    ws.check()
    got = y.cpu().numpy().T.astype(np.float64)
    assert np.array_equal(got[finite], O.bf16_to_f64(w)[finite][:, :8])
    assert np.isnan(got[~finite]).any(axis=1).all()  # 0 * inf or a NaN in the row


@pytest.mark.parametrize("act", sorted(uw.ACTIVATIONS))
def test_activations_over_their_range(act):
    """W = identity: y = act(x) for every BF16 x of up to 2^7, both signs."""
    import torch
    bits = np.arange(0x4300, dtype=np.uint16)  # 0 .. 128
    x = np.concatenate([bits, bits | 0x8000])
    x = np.resize(x, -(-x.size // 64) * 64).reshape(-1, 64)
    dm = device_matrix(synth.f32_to_bf16_bits(np.eye(64, dtype=np.float32)))
    y = torch.empty(x.shape[0], 64, dtype=torch.float32, device="cuda")
    ws = uw.Workspace(uw.epilogue_workspace_bytes(dm, x.shape[0]))
    uw.gemm_epilogue(dm, to_dev(x), y, ws, activation=act)
    ws.check()
    ref, bound = epilogue_bound(bf16_f64(x), 0.0, 0.0, act, 0.0, False)
    assert np.all(np.abs(y.cpu().numpy().astype(np.float64) - ref) <= bound)


@pytest.mark.parametrize("act", sorted(uw.ACTIVATIONS))
def test_activations_keep_their_relative_accuracy(act):
    """The same products against bounds relative to the activation: the tails
    of negative values, down to the smallest normal number."""
    import torch
    bits = np.arange(0x0080, 0x4300, dtype=np.uint16)  # 2^-126 .. 128
    x = np.concatenate([bits, bits | 0x8000])
    x = np.resize(x, -(-x.size // 64) * 64).reshape(-1, 64)
    dm = device_matrix(synth.f32_to_bf16_bits(np.eye(64, dtype=np.float32)))
    y = torch.empty(x.shape[0], 64, dtype=torch.float32, device="cuda")
    ws = uw.Workspace(uw.epilogue_workspace_bytes(dm, x.shape[0]))
    uw.gemm_epilogue(dm, to_dev(x), y, ws, activation=act)
    ws.check()
    v = bf16_f64(x)
    off = np.abs(y.cpu().numpy().astype(np.float64) - act_tail(v, act)) / activation_bound(v, act)
    assert off.max() <= 1, (float(off.max()), float(v.ravel()[off.argmax()]))


def test_swiglu_over_the_range_of_the_gate():
    """Gate = identity, up = 2^20 times it: h = SiLU(x) x 2^20 for every BF16 x
    of up to 128.  Relative error of SiLU in units of 2^-24: a fast exponential
    is off by 4 + 2.4 |x| at most (2 + 1.173 |x| units in the last place), its
    argument's rounding by |x| and a few for a scale; the divisor and the
    products take 1 to 4 each; BF16 rounds once more."""
    eye = np.eye(64, dtype=np.float32)
    gate, up = (experts_of([synth.f32_to_bf16_bits(m)]) for m in (eye, eye * 2.0 ** 20))
    bits = np.arange(0x0080, 0x4300, dtype=np.uint16)
    x = np.concatenate([bits, bits | 0x8000])
    x = np.resize(x, -(-x.size // 64) * 64).reshape(-1, 64)
    h = empty_bf16(*x.shape)
    ws = uw.Workspace(uw.grouped_workspace_bytes(gate, x.shape[0], swiglu=True))
    uw.gemm_grouped_swiglu(gate, up, to_dev(x), to_dev(offsets_of([x.shape[0]])), h, ws)
    ws.check()
    v = bf16_f64(x)
    silu = act_tail(v, "silu")
    ref = silu * v * 2.0 ** 20
    rel = np.minimum((13 + 3.6 * np.abs(v)) * F32, 1.0)
    # (a SiLU below the smallest normal number is held to that only)
    d = rel * np.abs(ref) + SMALLEST_NORMAL * np.abs(v) * 2.0 ** 20
    bound = d + HALF_ULP * (np.abs(ref) + d) + 2.0 ** -133
    off = np.abs(bf16_f64(to_host_u16(h)) - ref) / bound
    assert off.max() <= 1, (float(off.max()), float(v.ravel()[off.argmax()]))


# --------------------------- streams and workspaces --------------------------

def test_two_streams_with_their_own_workspaces():
    import torch
    mats = expert_weights(4, 1024, 2048, 960)
    ex = experts_of(mats)
    off = to_dev(offsets_of([5, 40, 0, 19]))
    xs = [to_dev(synth.activations(64, 2048, 961 + i)) for i in range(2)]
    want = []
    for x in xs:
        y, ws = empty_bf16(64, 1024), uw.Workspace(uw.grouped_workspace_bytes(ex, 64))
        uw.gemm_grouped(ex, x, off, y, ws, activation="silu")
        ws.check()
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    wss = [uw.Workspace(uw.grouped_workspace_bytes(ex, 64)) for _ in xs]
    outs = [empty_bf16(64, 1024) for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, y, ws in zip(streams, xs, outs, wss):
            uw.gemm_grouped(ex, x, off, y, ws, activation="silu", stream=s)
    torch.cuda.synchronize()
    for y, w, ws in zip(outs, want, wss):
        ws.check()
        assert torch.equal(y, w)


def test_one_workspace_for_calls_of_many_sizes():
    """The regions start at the same offsets for every call: products of
    different shapes, and the dense GEMM, take turns on one workspace."""
    import torch
    mats = expert_weights(3, 1024, 2048, 970)
    ex = experts_of(mats)
    dm = ex.matrices[0]
    ws = uw.Workspace(max(uw.grouped_workspace_bytes(ex, 300, swiglu=True), uw.workspace_bytes(dm, uw.PIPE_DIRECT, 100)))
    results = {}
    for turn in range(3):
        for n in (1, 300, 7, 64, 150):
            off = to_dev(offsets_of([n // 3, 0, n - n // 3]))
            x = to_dev(synth.activations(n, 2048, 971))
            y, h, g = empty_bf16(n, 1024), empty_bf16(n, 1024), empty_bf16(min(n, 100), 1024)
            uw.gemm_grouped(ex, x, off, y, ws)
            uw.gemm_grouped_swiglu(ex, ex, x, off, h, ws)
            uw.gemm_direct_palette(dm, x[:100], g, ws)
            ws.check()
            out = [to_host_u16(t) for t in (y, h, g)]
            if turn == 0:
                results[n] = out
            else:
                assert all(np.array_equal(a, b) for a, b in zip(out, results[n])), n


# --------------------------------- refusals ----------------------------------

def test_refusals_launch_nothing():
    import torch
    ex = experts_of(expert_weights(2, 128, 128, 980))
    other = experts_of(expert_weights(2, 256, 128, 982))
    x, y = empty_bf16(6, 128), empty_bf16(6, 128)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, 6, swiglu=True))
    small = uw.Workspace(1024)
    dm = ex.matrices[0]
    bad = [
        lambda: uw.gemm_grouped(ex, x[:, :64], off, y, ws),                       # columns
        lambda: uw.gemm_grouped(ex, empty_bf16(128, 6).t(), off, y, ws),          # not contiguous
        lambda: uw.gemm_grouped(ex, x.float(), off, y, ws),                       # type
        lambda: uw.gemm_grouped(ex, x.cpu(), off, y, ws),                         # device
        lambda: uw.gemm_grouped(ex, x, off.long(), y, ws),
        lambda: uw.gemm_grouped(ex, x, off[:2], y, ws),
        lambda: uw.gemm_grouped(ex, x, off, y.double(), ws),
        lambda: uw.gemm_grouped(ex, x[:5].contiguous(), off, y, ws),              # fewer rows of x than slots
        lambda: uw.gemm_grouped(ex, x, off, y, ws, rows=off),
        lambda: uw.gemm_grouped(ex, x, off, y, ws, bias=empty_bf16(128)),
        lambda: uw.gemm_grouped(ex, x, off, y, ws, residual=empty_bf16(6, 64)),
        lambda: uw.gemm_grouped(ex, x, off, y, ws, activation="swish"),
        lambda: uw.gemm_grouped(ex, x, off, y, small),
        lambda: uw.gemm_grouped_swiglu(ex, other, x, off, y, ws),
        lambda: uw.gemm_grouped_swiglu(ex, ex, x, off, empty_bf16(6, 64), ws),
        lambda: uw.gemm_epilogue(dm, x, y, small),
        lambda: uw.gemm_epilogue(dm, x, empty_bf16(5, 128), ws),
        lambda: uw.gemm_epilogue(dm, x, y, ws, bias=empty_bf16(1, 128)),
        lambda: uw.Experts([dm, other.matrices[0]]),
        lambda: uw.Experts([uw.DeviceMatrix(uw.encode(synth.weight_matrix(128, 128, 0.02, 0.0, 1.0, 1)))]),  # no pack
    ]
    n = uw.launch_count()
    for i, call in enumerate(bad):
        with pytest.raises(uw.UwError):
            call()
            pytest.fail(f"refusal {i}")
    assert uw.launch_count() == n
