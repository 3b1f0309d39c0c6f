"""GPU: router, weighted combination and the sparse MLP block against float64
forms written from their definitions."""
import math

import numpy as np
import pytest

from mlp_huffman_coded_b200 import synth
from mlp_huffman_coded_b200 import uw
from oracle import uw_oracle as O

from gpu_util import bf16_f64, device_matrix, empty_bf16, to_dev, to_host_u16
from moe_util import F32, HALF_ULP, expert_weights, product, route_ref, sum_bound

pytestmark = pytest.mark.gpu


def run_route(logits, k, renormalize=True, bf16=False):
    import torch
    T, E = logits.shape
    l = torch.from_numpy(np.ascontiguousarray(logits, dtype=np.float32)).cuda()
    r = uw.Route(T, E, k)
    r.rows.fill_(-7)
    ws = uw.Workspace(uw.route_workspace_bytes(T, E, k))
    uw.moe_route(l.to(torch.bfloat16) if bf16 else l, r, ws, renormalize=renormalize)
    ws.check("route")
    return r


def check_route(r, logits, k, renormalize=True):
    w, e, s, rows, off = route_ref(logits, k, renormalize)
    assert np.array_equal(r.experts.cpu().numpy(), e)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.slots.cpu().numpy(), s)
    n = int(off[-1])
    got = r.rows.cpu().numpy()
    assert np.array_equal(got[:n], rows)
    assert np.all(got[n:] == -7)  # entries past the last slot stay as they were
    # expf is off by at most 2 units in the last place plus its argument's
    # rounding (2^-24 |l - max|, and a weight with |l - max| > 88 is below
    # any that matters: 1e-38); the sum adds E roundings, the quotient one
    bound = (len(logits[0]) + 8 + 2 * 88) * F32 * w + 1e-37
    assert np.all(np.abs(r.weights.cpu().numpy().astype(np.float64) - w) <= bound)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 129, 700])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (8, 2), (33, 5), (64, 8), (130, 3), (256, 8), (40, 32), (200, 31), (1000, 32)])
def test_route_against_float64(T, E, k):
    logits = np.random.default_rng(T * 1000 + E).standard_normal((T, E)).astype(np.float32) * 2
    for ren in (True, False):
        check_route(run_route(logits, k, ren), logits, k, ren)


@pytest.mark.parametrize("T", [1, 64, 65, 700])
@pytest.mark.parametrize("E,k", [(9, 2), (16, 3), (17, 4), (32, 8), (65, 8), (128, 8), (129, 8), (257, 8), (1024, 32)])
def test_route_on_both_sides_of_every_width(T, E, k):
    """A lane's logits are 1, 2, 4, .. 32 of a token's: the borders between
    them, and the largest router, with one block and with several."""
    logits = np.random.default_rng(T * 2000 + E).standard_normal((T, E)).astype(np.float32) * 2
    logits[T // 2, : E - 1] = -np.inf  # one expert left, the last
    for ren in (True, False):
        check_route(run_route(logits, k, ren), logits, k, ren)


def test_route_bf16_logits_tie_often():
    logits = synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(
        np.round(np.random.default_rng(3).standard_normal((300, 40)) * 4).astype(np.float32)))
    logits[5] = 0.0
    logits[6, ::2] = -0.0
    check_route(run_route(logits, 6, bf16=True), logits, 6)


def test_route_masked_rows_infinities_and_nans():
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((200, 16)).astype(np.float32)
    low = np.finfo(np.float32).min
    logits[3] = -np.inf                       # nothing left
    logits[4, 1:] = -np.inf                   # one expert left
    logits[5] = np.nan
    logits[6, ::3] = np.nan
    logits[7, 2] = logits[7, 9] = np.inf      # share the weight
    logits[8] = low                           # the type's lowest value is a value
    logits[9, :8] = low
    logits[150:] = -np.inf                    # a padded batch
    for ren in (True, False):
        check_route(run_route(logits, 4, ren), logits, 4, ren)


def test_route_every_token_to_one_expert_and_none_at_all():
    logits = np.full((500, 12), -np.inf, np.float32)
    check_route(run_route(logits, 2), logits, 2)
    logits[:, 7] = 1.0
    check_route(run_route(logits, 2), logits, 2)


def test_route_no_tokens():
    r = uw.Route(0, 8, 2)
    r.offsets.fill_(5)
    ws = uw.Workspace(uw.route_workspace_bytes(0, 8, 2))
    import torch
    uw.moe_route(torch.empty(0, 8, device="cuda"), r, ws)
    ws.check()
    assert r.offsets.tolist() == [0] * 9


def test_route_more_tokens_than_one_chunk_per_block():
    """20000 tokens: every block ranks several runs of 64."""
    logits = np.random.default_rng(5).standard_normal((20000, 8)).astype(np.float32)
    check_route(run_route(logits, 2), logits, 2)


# ------------------------------- combine -------------------------------------

def combine_check(parts, slots, weights, residual, y, bf16_parts):
    p = O.bf16_to_f64(parts) if bf16_parts else parts.astype(np.float64)
    n = p.shape[0]
    T, k = slots.shape
    ref = np.zeros((T, p.shape[1])) if residual is None else O.bf16_to_f64(residual).copy()
    size = np.abs(ref)
    for j in range(k):
        for t in range(T):
            if 0 <= slots[t, j] < n:
                v = float(weights[t, j]) * p[slots[t, j]]
                ref[t] += v
                size[t] += np.abs(v)
    d = (k + 1) * F32 * size  # k fused multiply-adds and one addition
    d = d + HALF_ULP * (np.abs(ref) + d) + 1e-38
    assert np.all(np.abs(y - ref) <= d)


@pytest.mark.parametrize("cols", [1, 7, 8, 264, 2048, 4100])
@pytest.mark.parametrize("T,k", [(1, 1), (3, 2), (65, 5), (40, 9)])
@pytest.mark.parametrize("bf16_parts", [False, True])
def test_combine_against_float64(cols, T, k, bf16_parts):
    import torch
    rng = np.random.default_rng(cols + T)
    n = T * k
    parts = rng.standard_normal((n, cols)).astype(np.float32)
    if bf16_parts:
        parts = synth.f32_to_bf16_bits(parts)
    slots = rng.permutation(n).reshape(T, k).astype(np.int32)
    slots[0, 0] = -1
    if T > 2:
        slots[2] = -1        # no expert at all: the residual, or zero
        slots[1, 1] = n      # outside: adds nothing
        slots[1, 0] = slots[0, 1]
    weights = rng.random((T, k)).astype(np.float32)
    weights[0, 0] = np.nan   # of a slot that is not there
    res = synth.activations(T, cols, 7)
    for r in (None, res):
        y = empty_bf16(T, cols)
        uw.moe_combine(to_dev(parts), to_dev(slots), torch.from_numpy(weights).cuda(), y,
                       residual=None if r is None else to_dev(r))
        combine_check(parts, slots, weights, r, bf16_f64(to_host_u16(y)), bf16_parts)
    r = to_dev(res)
    uw.moe_combine(to_dev(parts), to_dev(slots), torch.from_numpy(weights).cuda(), r, residual=r)
    assert np.array_equal(to_host_u16(r), to_host_u16(y))  # in place


def test_combine_of_unaligned_slices():
    import torch
    T, k, cols = 6, 2, 256
    rng = np.random.default_rng(8)
    parts = rng.standard_normal((T * k, cols)).astype(np.float32)
    res = synth.activations(T, cols, 9)
    slots = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    weights = rng.random((T, k)).astype(np.float32)

    def shifted(t):  # the same values one element into a larger tensor
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    y = shifted(empty_bf16(T, cols))
    uw.moe_combine(shifted(to_dev(parts)), shifted(to_dev(slots)), shifted(torch.from_numpy(weights).cuda()), y,
                   residual=shifted(to_dev(res)))
    combine_check(parts, slots, weights, res, bf16_f64(to_host_u16(y)), False)


# -------------------------------- block --------------------------------------

def block_ref(gs, us, ds, x, logits, k, residual, renormalize=True):
    """(y, bound): h rounded to BF16 once (HALF_ULP), sums as bounded for the
    single products, weights within the router's bound."""
    w, e, _, _, _ = route_ref(logits, k, renormalize)
    T, d = x.shape
    ref = np.zeros((T, d)) if residual is None else O.bf16_to_f64(residual).copy()
    bound = F32 * np.abs(ref)
    for t in range(T):
        for j in range(k):
            if e[t, j] < 0:
                continue
            xt = x[t:t + 1]
            g, ag = product(gs[e[t, j]], xt)
            u, au = product(us[e[t, j]], xt)
            K = x.shape[1]
            dg, du = sum_bound(ag, K), sum_bound(au, K)
            s = O.silu(g)
            h = s * u
            dh = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + 16 * F32 * (np.abs(g) + np.abs(s)) * np.abs(u)
            dh = dh + HALF_ULP * (np.abs(h) + dh)
            wd = O.bf16_to_f64(ds[e[t, j]])
            part = (h @ wd.T)[0]
            ab = ((np.abs(h) + dh) @ np.abs(wd).T)[0]
            dpart = (dh @ np.abs(wd).T)[0] + sum_bound(ab, wd.shape[1])
            dw = (logits.shape[1] + 8 + 176) * F32 * w[t, j]
            ref[t] += w[t, j] * part
            bound[t] += w[t, j] * dpart + dw * (np.abs(part) + dpart) + 4 * F32 * w[t, j] * (np.abs(part) + dpart)
    bound = bound + (k + 1) * F32 * np.abs(ref)
    return ref, bound + HALF_ULP * (np.abs(ref) + bound) + 1e-30


def experts_of(mats):
    return uw.Experts([device_matrix(m) for m in mats])


@pytest.fixture(scope="module")
def sparse_mlp():
    E, d, ffn = 6, 256, 320
    mats = expert_weights(E, ffn, d, 600), expert_weights(E, ffn, d, 620), expert_weights(E, d, ffn, 640)
    return mats, [experts_of(m) for m in mats]


@pytest.mark.parametrize("T", [1, 2, 17, 150])
@pytest.mark.parametrize("k", [1, 2, 6])
def test_block_against_float64(sparse_mlp, T, k):
    import torch
    (gs, us, ds), ex = sparse_mlp
    d = ds[0].shape[0]
    x = synth.activations(T, d, 660 + T)
    logits = np.random.default_rng(T).standard_normal((T, len(gs))).astype(np.float32)
    if T > 4:
        logits[3] = -np.inf   # padded token: the residual passes through
        logits[4, 1:] = -np.inf
    res = synth.activations(T, d, 661)
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    for r, ren in ((None, True), (res, False)):
        y = empty_bf16(T, d)
        uw.moe_block(*ex, to_dev(x), torch.from_numpy(logits).cuda(), k, y, ws,
                     residual=None if r is None else to_dev(r), renormalize=ren)
        ws.check("block")
        ref, bound = block_ref(gs, us, ds, x, logits, k, r, ren)
        got = bf16_f64(to_host_u16(y))
        assert np.all(np.abs(got - ref) <= bound), float(np.max(np.abs(got - ref) - bound))


def test_block_of_padded_tokens_only(sparse_mlp):
    import torch
    _, ex = sparse_mlp
    T, k, d = 20, 2, ex[2].rows
    x, res = to_dev(synth.activations(T, d, 665)), to_dev(synth.activations(T, d, 666))
    logits = torch.full((T, len(ex[0])), -math.inf, device="cuda")
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    y, z = empty_bf16(T, d), empty_bf16(T, d)
    uw.moe_block(*ex, x, logits, k, y, ws, residual=res)
    uw.moe_block(*ex, x, logits, k, z, ws)
    ws.check()
    assert torch.equal(y, res) and not bool(z.any())


def test_block_equals_its_four_calls(sparse_mlp):
    import torch
    _, ex = sparse_mlp
    T, k, d, ffn = 45, 2, ex[2].rows, ex[0].rows
    x = to_dev(synth.activations(T, d, 670))
    res = to_dev(synth.activations(T, d, 671))
    logits = torch.randn(T, len(ex[0]), device="cuda")
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    y = empty_bf16(T, d)
    uw.moe_block(*ex, x, logits, k, y, ws, residual=res)
    r = uw.Route(T, len(ex[0]), k)
    h, parts, y2 = empty_bf16(T * k, ffn), torch.empty(T * k, d, device="cuda"), empty_bf16(T, d)
    uw.moe_route(logits, r, ws)
    uw.gemm_grouped_swiglu(ex[0], ex[1], x, r.offsets, h, ws, rows=r.rows)
    uw.gemm_grouped(ex[2], h, r.offsets, parts, ws)
    uw.moe_combine(parts, r.slots, r.weights, y2, residual=res)
    ws.check()
    assert torch.equal(y, y2)


def test_a_workspace_for_the_largest_batch_serves_smaller_ones(sparse_mlp):
    import torch
    _, ex = sparse_mlp
    E, d, k = len(ex[0]), ex[2].rows, 2
    big = uw.Workspace(uw.moe_workspace_bytes(*ex, 400, k))
    for T in (400, 1, 30, 33, 70, 129, 200, 399):
        x, logits = to_dev(synth.activations(T, d, 680)), torch.randn(T, E, device="cuda")
        y, z = empty_bf16(T, d), empty_bf16(T, d)
        own = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
        uw.moe_block(*ex, x, logits, k, y, big)
        uw.moe_block(*ex, x, logits, k, z, own)
        big.check()
        own.check()
        assert torch.equal(y, z), T


def test_layers_chained_on_one_stream_match_layers_one_by_one(sparse_mlp):
    """Launches overlap (a kernel starts while the one before it finishes);
    ten blocks in a row, in place on the residual stream, equal the same
    blocks with the device idle between them, and a dense product that
    follows sees the last one's output."""
    import torch
    _, ex = sparse_mlp
    T, k, d = 9, 2, ex[2].rows
    x0 = to_dev(synth.activations(T, d, 680))
    logits = torch.randn(10, T, len(ex[0]), device="cuda")
    dm = device_matrix(synth.weight_matrix(384, d, 0.02, 1e-3, 200.0, 681))
    ws = uw.Workspace(max(uw.moe_workspace_bytes(*ex, T, k), uw.workspace_bytes(dm, uw.PIPE_DIRECT, T)))

    def chain(sync):
        x, y = x0.clone(), empty_bf16(T, 384)
        for l in logits:
            uw.moe_block(*ex, x, l, k, x, ws, residual=x)
            if sync:
                torch.cuda.synchronize()
        uw.gemm_direct_palette(dm, x, y, ws)
        ws.check()
        return x, y

    slow = chain(True)
    for _ in range(5):
        fast = chain(False)
        assert torch.equal(fast[0], slow[0]) and torch.equal(fast[1], slow[1])


@pytest.mark.parametrize("T", [9, 30, 150, 700])
def test_every_call_of_a_chain_sees_its_own_routing(sparse_mlp, T):
    """Twelve blocks in a row on one workspace, each with a routing of its
    own, against the same calls with the device idle between them.  From 9
    tokens on the rows of x are copied next to each other first, so both
    products read the groups before they wait for the kernel ahead."""
    import torch
    _, ex = sparse_mlp
    k, d, E, n = 2, ex[2].rows, len(ex[0]), 12
    x = to_dev(synth.activations(T, d, 685))
    g = torch.Generator(device="cuda").manual_seed(T)
    # each call prefers other experts: groups of very different sizes
    logits = torch.randn(n, T, E, device="cuda", generator=g) + 4 * torch.randn(n, 1, E, device="cuda", generator=g)
    logits[5] = -math.inf  # no group has a slot
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))

    def chain(sync):
        ys = [empty_bf16(T, d) for _ in range(n)]
        for l, y in zip(logits, ys):
            uw.moe_block(*ex, x, l, k, y, ws)
            if sync:
                torch.cuda.synchronize()
        ws.check()
        return ys

    slow = chain(True)
    assert not bool(slow[5].any()) and not torch.equal(slow[0], slow[1])
    for _ in range(5):
        for a, b in zip(chain(False), slow):
            assert torch.equal(a, b)


def test_captured_block_replays_on_new_inputs(sparse_mlp):
    """Routing is on the device, so one captured graph serves every batch of
    its size, whatever its groups; on another stream than the default."""
    import torch
    _, ex = sparse_mlp
    T, k, d, E = 12, 2, ex[2].rows, len(ex[0])
    side = torch.cuda.Stream()
    x, l, y = empty_bf16(T, d), torch.empty(T, E, device="cuda"), empty_bf16(T, d)
    with torch.cuda.stream(side):
        ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
        x.zero_()
        l.zero_()
        uw.moe_block(*ex, x, l, k, y, ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            uw.moe_block(*ex, x, l, k, y, ws)
    for seed in range(4):
        x.copy_(to_dev(synth.activations(T, d, 690 + seed)))
        l.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32) * (1 + 4 * seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = empty_bf16(T, d)
        uw.moe_block(*ex, x, l, k, want, ws)
        ws.check()
        assert torch.equal(y, want)


def test_graphs_of_several_blocks_share_a_workspace(sparse_mlp):
    """Two captured graphs of four blocks each, on one workspace, replayed in
    turn without a pause."""
    import torch
    _, ex = sparse_mlp
    T, k, d, E = 70, 2, ex[2].rows, len(ex[0])
    side = torch.cuda.Stream()
    x = to_dev(synth.activations(T, d, 695))
    logits = torch.randn(2, 4, T, E, device="cuda") + 3 * torch.randn(2, 4, 1, E, device="cuda")
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    want = [empty_bf16(T, d) for _ in range(8)]
    for l, y in zip(logits.view(8, T, E), want):
        uw.moe_block(*ex, x, l, k, y, ws, residual=x)
        torch.cuda.synchronize()
    got = [empty_bf16(T, d) for _ in range(8)]
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for l, y in zip(logits[i], got[4 * i:4 * i + 4]):
                uw.moe_block(*ex, x, l, k, y, ws, residual=x)
        graphs.append(graph)
    for _ in range(5):
        for y in got:
            y.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        ws.check()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_products_take_unaligned_slices(sparse_mlp):
    """Bias, residual, offsets and row numbers one element into larger
    tensors (x, y and the workspace are 16-byte aligned)."""
    import torch
    _, ex = sparse_mlp
    E, n, ffn, d = len(ex[0]), 50, ex[0].rows, ex[0].cols

    def shifted(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    x = to_dev(synth.activations(30, d, 696))
    bias, res = to_dev(synth.activations(E, ffn, 697)), to_dev(synth.activations(n, ffn, 698))
    off = torch.tensor([0, 20, 20, 23, 40, 41, 50], dtype=torch.int32, device="cuda")
    rows = torch.randint(0, 30, (n,), dtype=torch.int32, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex[0], n))
    for fp32 in (False, True):
        y = torch.zeros(n, ffn, dtype=torch.float32 if fp32 else torch.bfloat16, device="cuda")
        z = torch.zeros_like(y)
        uw.gemm_grouped(ex[0], x, off, y, ws, rows=rows, bias=bias, activation="gelu_tanh", residual=res)
        uw.gemm_grouped(ex[0], x, shifted(off), z, ws, rows=shifted(rows), bias=shifted(bias), activation="gelu_tanh",
                        residual=shifted(res))
        ws.check()
        assert torch.equal(y, z) and bool(y.any())


def test_route_of_a_million_tokens():
    import torch
    T, E, k = 1 << 20, 8, 3
    g = torch.Generator(device="cuda").manual_seed(6)
    logits = torch.argsort(torch.rand(T, E, device="cuda", generator=g), dim=1).float()  # 0 .. 7 in any order: no ties
    logits[::5] = -math.inf
    r = uw.Route(T, E, k)
    ws = uw.Workspace(uw.route_workspace_bytes(T, E, k))
    uw.moe_route(logits, r, ws)
    ws.check()
    chosen = torch.topk(logits, k, dim=1).indices.int()
    chosen[::5] = -1
    assert torch.equal(r.experts, chosen)
    flat = torch.where(chosen < 0, E, chosen).flatten()
    order = torch.sort(flat, stable=True).indices
    n = int((flat < E).sum())
    assert torch.equal(r.rows[:n].long(), order[:n] // k)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    assert r.offsets.tolist() == [0] + torch.cumsum(counts, 0).tolist()
    slots = torch.full_like(flat, -1)
    slots[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(r.slots.flatten(), slots)


# the sizes of the framework's own blocks: waves, shared tiles, rows laid next to
# each other, and row-tile pairs in the down product

@pytest.fixture(scope="module")
def full_size_mlp():
    import torch
    E, d, ffn = 8, 4096, 14336
    load = uw.Workspace(256)

    def experts(rows, cols, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        mats = [(torch.randn(rows, cols, generator=g, device="cuda") * 0.02).to(torch.bfloat16) for _ in range(E)]
        return mats, uw.Experts([uw.DeviceMatrix.encode_on_device(w).prepare_direct_palette(load, keep_idx4=False)
                                 for w in mats])

    made = [experts(ffn, d, 710), experts(ffn, d, 711), experts(d, ffn, 712)]
    yield [m for m, _ in made], [e for _, e in made]
    del made
    torch.cuda.empty_cache()


def full_size_inputs(T, seed, E=8, d=4096):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
    if T > 4:
        logits[2] = -math.inf  # a padded token
    return x, logits


@pytest.mark.parametrize("T", [1, 32, 600])
def test_full_size_block_against_float64(full_size_mlp, T):
    import torch
    (gs, us, ds), ex = full_size_mlp
    x, logits = full_size_inputs(T, 720 + T)
    k, E, K, F = 2, 8, 4096, 14336
    res = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    y = torch.empty_like(x)
    uw.moe_block(*ex, x, logits, k, y, ws, residual=res)
    ws.check()
    w, chosen, _, _, _ = route_ref(logits.cpu().numpy(), k)
    w, chosen = torch.from_numpy(w).cuda(), torch.from_numpy(chosen).cuda()
    xd, ref = x.double(), res.double()
    bound = F32 * ref.abs()
    for e in range(E):  # as block_ref, expert by expert
        t, j = torch.nonzero(chosen == e, as_tuple=True)
        if not t.numel():
            continue
        g, ag = xd[t] @ gs[e].double().T, xd[t].abs() @ gs[e].double().abs().T
        u, au = xd[t] @ us[e].double().T, xd[t].abs() @ us[e].double().abs().T
        dg, du = K * 2.0 ** -23 * ag, K * 2.0 ** -23 * au
        s = g / (1 + torch.exp(-g))
        h = s * u
        dh = 1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + 16 * F32 * (g.abs() + s.abs()) * u.abs()
        dh = dh + HALF_ULP * (h.abs() + dh)
        part, ab = h @ ds[e].double().T, (h.abs() + dh) @ ds[e].double().abs().T
        dpart = dh @ ds[e].double().abs().T + F * 2.0 ** -23 * ab
        wt = w[t, j][:, None]
        ref.index_add_(0, t, wt * part)
        bound.index_add_(0, t, wt * dpart + (E + 184) * F32 * wt * (part.abs() + dpart) + 4 * F32 * wt * (part.abs() + dpart))
    bound = bound + (k + 1) * F32 * ref.abs()
    bound = bound + HALF_ULP * (ref.abs() + bound) + 1e-30
    off = (y.double() - ref).abs()
    assert float((off - bound).max()) <= 0
    # the bounds add up worst cases of every sum; over all values the roundings
    # of h and y count, each at most 2^-8 / sqrt(3) in the mean square
    assert float(off.pow(2).mean().sqrt() / ref.pow(2).mean().sqrt()) <= HALF_ULP
    if T > 4:
        assert torch.equal(y[2], res[2])


@pytest.mark.parametrize("T", [1, 32, 600])
def test_full_size_blocks_in_a_row_equal_their_four_calls(full_size_mlp, T):
    """Six blocks without a pause between them, each with a routing of its
    own, against the four calls one by one with the device idle in between."""
    import torch
    _, ex = full_size_mlp
    k, E, d, ffn = 2, 8, 4096, 14336
    inputs = [full_size_inputs(T, 730 + i) for i in range(6)]
    ws = uw.Workspace(uw.moe_workspace_bytes(*ex, T, k))
    r = uw.Route(T, E, k)
    h, parts = torch.empty(T * k, ffn, dtype=torch.bfloat16, device="cuda"), torch.empty(T * k, d, device="cuda")
    want = []
    for x, l in inputs:
        y = torch.empty_like(x)
        for call in (lambda: uw.moe_route(l, r, ws), lambda: uw.gemm_grouped_swiglu(ex[0], ex[1], x, r.offsets, h, ws, rows=r.rows),
                     lambda: uw.gemm_grouped(ex[2], h, r.offsets, parts, ws), lambda: uw.moe_combine(parts, r.slots, r.weights, y)):
            call()
            torch.cuda.synchronize()
        want.append(y)
    ws.check()
    for _ in range(3):
        got = [torch.empty_like(x) for x, _ in inputs]
        for (x, l), y in zip(inputs, got):
            uw.moe_block(*ex, x, l, k, y, ws)
        ws.check()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------- refusals on the device ----------------------------

@pytest.mark.parametrize("offsets", [[0, 5, 3, 8], [-1, 2, 3, 8], [0, 2, 3, 9], [9, 9, 9, 9]])
def test_bad_offsets_are_reported_and_nothing_is_computed(offsets):
    import torch
    ex = experts_of(expert_weights(3, 128, 128, 700))
    x = to_dev(synth.activations(8, 128, 701))
    y = torch.full((8, 128), 3.0, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, 8))
    uw.gemm_grouped(ex, x, torch.tensor(offsets, dtype=torch.int32, device="cuda"), y, ws)
    assert ws.status() == uw.UW_ERR_INVALID_ARG
    assert bool((y == 3.0).all())
    good = torch.tensor([0, 2, 3, 8], dtype=torch.int32, device="cuda")
    uw.gemm_grouped(ex, x, good, y, ws)
    ws.check("after")


def test_a_row_number_outside_x_is_reported():
    import torch
    mats = expert_weights(2, 128, 128, 710)
    ex = experts_of(mats)
    x = to_dev(synth.activations(4, 128, 711))
    y = torch.zeros(6, 128, device="cuda")
    ws = uw.Workspace(uw.grouped_workspace_bytes(ex, 6))
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 1, 2, 3, 0, 1], dtype=torch.int32, device="cuda")
    uw.gemm_grouped(ex, x, off, y, ws, rows=good)
    ws.check()
    for bad in (4, -1, 2**31 - 1, -2**31):
        r, z = good.clone(), torch.zeros_like(y)
        r[4] = bad
        uw.gemm_grouped(ex, x, off, z, ws, rows=r)
        assert ws.status() == uw.UW_ERR_INVALID_ARG
        keep = torch.arange(6, device="cuda") != 4
        assert torch.equal(z[keep], y[keep])  # the other slots are right
