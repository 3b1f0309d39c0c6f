"""GPU: products grouped by expert and products with a fused epilogue,
against float64 at group sizes, shapes and epilogues where they can go
wrong."""
import numpy as np
import pytest

from mlp_huffman_coded_b200 import synth
from mlp_huffman_coded_b200 import uw
from oracle import uw_oracle as O

from gpu_util import bf16_f64, device_matrix, empty_bf16, to_dev, to_host_u16
from moe_util import check_slots, expert_weights, grouped_ref, swiglu_ref

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


@pytest.mark.parametrize("batch", [1, 16, 17, 100, 256, 257, 600])
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
