"""The key-value cache in 4 bits and the page pool on the GPU against the oracle."""
import numpy as np
import pytest
import torch

import kv4_cases
import kv_cases
from dynamic_tree_speculative_gb300 import binding as B
from oracle import kv4_oracle as O4
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _nodes(c):
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return None if c.parent is None and c.n_nodes is None else B.NodeArrays(up(c.parent), up(c.depth), up(c.n_nodes))


def _cache4(c, codes=None, layout="head"):
    """The case's cache, quantised by the oracle (or `codes`: key codes, value codes, scale)."""
    k, v, scale = (kv4_cases.quantised(c) if codes is None else codes)[:3]
    there = lambda x: x.cuda() if layout == "token" else x.transpose(2, 3).contiguous().cuda().transpose(2, 3)  # noqa: E731
    return B.KVCache4(there(k), there(v), scale.cuda(), c.table.cuda(), c.seq_len.cuda())


def _cache(c):
    return B.KVCache(c.k.contiguous().cuda(), c.v.contiguous().cuda(), c.table.cuda(), c.seq_len.cuda())


def _queries(seed, c, Hq, gain=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((len(c.counts), c.N, Hq, c.k.shape[4]), generator=g) * gain).to(c.dtype)


def _run_attend(c, q, scale=None, layer=0, ws=None, cache=None, layout="head"):
    cache = cache or _cache4(c, layout=layout)
    qd = q.cuda()
    out = torch.full(qd.shape, NAN, dtype=c.dtype, device="cuda")
    ws = ws or B.AttendWorkspace(cache.B, c.N, q.shape[2], c.k.shape[3], c.k.shape[4])
    status = _status()
    B.spec_tree_kv4_attend(cache, layer, qd, out, ws, status, tree=_nodes(c), node_begin=c.begin, scale=scale)
    torch.cuda.synchronize()
    return out.cpu(), int(status.item())


def _expected(c, q, codes, scale, layer=0):
    """The oracle's outputs over the values that the codes stand for, and the bound on the error."""
    _, _, sc, kp, vp = codes
    kp, vp = kp[layer], vp[layer]
    D, few = q.shape[3], c.N * (q.shape[2] // c.k.shape[3]) <= kv4_cases.FEW_ROWS
    parents = None if c.parent is None else c.parent.numpy()
    call = lambda qq, k, v: O.attend(qq, k, v, c.table.numpy(), c.seq_len.numpy(), parents, c.counts, c.begin, scale)  # noqa: E731
    (ks, km), (vs, vm) = (tuple(x[layer] for x in kv4_cases.steps(c, None, sc, w)) for w in (0, 1))
    qn = q.double().numpy()
    out, mean_v, _, _ = call(qn, kp, vp)
    wide = lambda x: np.repeat(x[..., None], D, -1)  # noqa: E731
    # sums over the tokens with the outputs' own weights: |v| + |middle| + |zero|, and 15 steps
    mean_m = call(qn, kp, wide(np.abs(vm) + np.abs(vm - 8 * vs)))[0]
    steps_v = call(qn, kp, wide(15 * np.abs(vs)))[0]
    # the largest scale * sum |q| x over what a row sees
    q_k = call(np.abs(qn), np.abs(kp), vp)[2]
    floor_k = call(np.abs(qn), np.full_like(kp, np.nanmax(np.abs(np.where(np.isfinite(kp), kp, 0)))), vp)[2]
    floor_v = np.nanmax(np.abs(np.where(np.isfinite(vp), vp, 0)))
    k_abs = call(np.abs(qn), wide(15 * np.abs(ks) + np.abs(km - 8 * ks)), vp)[2]
    tokens = int(c.seq_len.max()) + c.begin + c.N
    return out, kv4_cases.attend_bound(c.dtype, out, k_abs, q_k, floor_k, floor_v, mean_v + mean_m, steps_v, D, tokens, few)


def _check_attend(c, q, scale=None, layer=0, layout="head"):
    codes = kv4_cases.quantised(c)
    got, status = _run_attend(c, q, scale, layer, cache=_cache4(c, codes, layout))
    want, bound = _expected(c, q, codes, q.shape[3] ** -0.5 if scale is None else scale, layer)
    err = np.abs(got.double().numpy() - want)
    assert status == 0 and (err <= bound).all(), (status, float(np.nanmax(err / bound)), int((~(err <= bound)).sum()))
    # all roundings together, in the 2-norm: the output's half step h at most, and 2^-11 each of the weights, keys (times the
    # scores' spread, up to four) and values, of outputs that are at least a hundredth of the values
    if np.linalg.norm(want) > 0 and scale is None:
        h = kv_cases.half_step(c.dtype)
        assert np.linalg.norm(err) <= (h + 6 * 2.0 ** -11) * max(np.linalg.norm(want), 0.1 * np.sqrt(want.size))


# --------------------------------------------------------------- attention ---

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [5, 0, 127], [15, 16, 17, 31], [128, 129, 300], [1000, 3]])
def test_one_token(dtype, D, lens):
    c = kv_cases.make(1, lens, 1, 2, D, 16, dtype, tree=False, stale=NAN)
    _check_attend(c, _queries(2, c, 8))


@pytest.mark.parametrize("Hq,Hkv,N,dtype,D", [(1, 1, 1, "bf16", 128), (7, 1, 1, "f16", 128), (9, 1, 1, "bf16", 64),
                                              (16, 1, 1, "bf16", 128), (6, 6, 5, "bf16", 128), (4, 1, 4, "f16", 64),
                                              (8, 2, 4, "bf16", 128), (5, 1, 3, "bf16", 64), (17, 1, 1, "bf16", 128),
                                              (6, 6, 16, "bf16", 128), (6, 6, 17, "bf16", 128)])
def test_few_rows(Hq, Hkv, N, dtype, D):
    """Around the 8, 16 and more rows that a key head's heads make of a call's nodes."""
    c = kv_cases.make(3, [60, 0, 140], N, Hkv, D, 16, dtype, counts=[N, N, max(1, N - 2)], stale=NAN)
    _check_attend(c, _queries(4, c, Hq))


@pytest.mark.parametrize("lens", [[0], [3, 64, 130], [70, 515]])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (2, 2, 128, "f16"), (4, 4, 64, "bf16"),
                                            (7, 1, 64, "f16"), (10, 2, 128, "bf16")])
def test_tree(lens, Hq, Hkv, D, dtype):
    c = kv_cases.make(5, lens, 61, Hkv, D, 16, dtype, stale=INF)
    _check_attend(c, _queries(6, c, Hq))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("N,D", [(1, 128), (33, 128), (1, 64), (33, 64)])
def test_pages(page, layout, N, D):
    c = kv_cases.make(7, [200, 61, 7], N, 2, D, page, stale=NAN)
    _check_attend(c, _queries(8, c, 4), layout=layout)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 17, 64, 65, 127, 128, 129, 200])
def test_tree_sizes(n):
    c = kv_cases.make(9, [90, 40], n, 1, 64, 32, tree=True, counts=[n, max(1, n - 5)], stale=NAN)
    _check_attend(c, _queries(10, c, 3))


def test_largest_tree():
    c = kv_cases.make(11, [33], 512, 1, 64, 32)
    _check_attend(c, _queries(12, c, 2))


@pytest.mark.parametrize("begin,N", [(1, 8), (9, 8), (25, 8), (130, 6), (0, 1), (40, 2), (500, 3)])
@pytest.mark.parametrize("Hq", [2, 8])
def test_frontier(begin, N, Hq):
    """A drafter's frontier: the call's nodes come behind earlier ones, whose entries are in the cache."""
    c = kv_cases.make(13, [100, 31, 0], N, 2, 64, 16, begin=begin, counts=[begin + N, begin + N - 1, begin], stale=NAN)
    _check_attend(c, _queries(14, c, Hq))


@pytest.mark.parametrize("N,lens,Hq,Hkv", [(40, [0], 4, 1), (130, [77], 4, 2), (300, [10, 500], 2, 1), (600, [0], 1, 1),
                                           (3, [500, 2], 4, 1), (16, [300], 1, 1)])
def test_chunk(N, lens, Hq, Hkv):
    c = kv_cases.make(15, lens, N, Hkv, 128, 64, tree=False, stale=NAN)
    _check_attend(c, _queries(16, c, Hq))


def test_chain_begin_and_counts():
    for N, begin, counts in ((70, 30, [100, 41, 30]), (4, 30, [34, 31, 30])):
        c = kv_cases.make(17, [50, 9, 4], N, 1, 128, 16, tree=False, begin=begin, counts=counts, stale=NAN)
        _check_attend(c, _queries(18, c, 4))


def test_many_short_sequences():
    rng = np.random.RandomState(0)
    c = kv_cases.make(19, rng.randint(0, 60, 300).tolist(), 1, 1, 64, 8, tree=False, stale=NAN)
    _check_attend(c, _queries(20, c, 2))


@pytest.mark.parametrize("N", [1, 9])
def test_layers_and_scale(N):
    c = kv_cases.make(21, [140, 20], N, 2, 128, 16, layers=3, stale=NAN)
    for layer in (0, 2):
        _check_attend(c, _queries(22, c, 4), scale=0.31, layer=layer)
    _check_attend(c, _queries(22, c, 4), scale=0.0)
    _check_attend(c, _queries(22, c, 4), scale=-0.05)


@pytest.mark.parametrize("N", [1, 3, 12])
def test_sharp_scores(N):
    """Scores spread over hundreds: the running maximum moves by more than any threshold, both ways."""
    c = kv_cases.make(23, [700, 260], N, 1, 128, 16)
    for order in (1, -1):
        k = c.k.clone()
        for b, n in enumerate(c.seq_len.tolist()):
            for s in range(n):
                k[0, int(c.table[b, s // 16]), s % 16] *= (s if order > 0 else n - s) / 40.0
        c2 = kv_cases.dataclasses.replace(c, k=k)
        got, status = _run_attend(c2, _queries(24, c, 4))
        codes = kv4_cases.quantised(c2)
        want, bound = _expected(c2, _queries(24, c, 4), codes, 128 ** -0.5)
        assert status == 0 and (np.abs(got.double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("gain", [1e-20, 1e-6, 1e4, 1e30])
@pytest.mark.parametrize("N", [1, 40])
def test_values_of_any_size(gain, N):
    """Values far from one: scales of any size times the weights."""
    c = kv_cases.make(25, [300, 20], N, 1, 64, 16)
    _check_attend(kv_cases.dataclasses.replace(c, v=(c.v.double() * gain).to(c.dtype)), _queries(26, c, 4))


@pytest.mark.parametrize("Hq,N", [(8, 61), (2, 9)])
def test_unseen_nodes_have_no_influence(Hq, N):
    """NaN in nodes off the path (keys, values): their descendants get NaN, everyone else the same bits as without."""
    c = kv_cases.make(27, [37, 150], N, 2, 128, 16, stale=NAN)
    q = _queries(28, c, Hq)
    clean, _ = _run_attend(c, q)
    for what, value in (("v", NAN), ("v", INF), ("k", NAN), ("k", -INF)):
        hit = 5
        x = getattr(c, what).clone()
        for b in range(2):
            s = int(c.seq_len[b]) + hit
            x[0, int(c.table[b, s // 16]), s % 16] = value
        got, status = _run_attend(kv_cases.dataclasses.replace(c, **{what: x}), q)
        assert status == 0
        for b in range(2):
            for n in range(N):
                if hit in O.sees(c.parent[b].numpy(), n):
                    assert got[b, n].isnan().all(), (what, value, b, n)
                else:
                    assert torch.equal(got[b, n], clean[b, n]), (what, value, b, n)


@pytest.mark.parametrize("Hq,N,D", [(8, 4, 128), (2, 9, 64), (4, 4, 64), (8, 61, 128), (8, 8, 64), (2, 40, 128)])
@pytest.mark.parametrize("value", [INF, NAN, 3e38, -1e30])
def test_rows_have_no_influence_on_each_other(Hq, N, D, value):
    """What one node's queries hold leaves the others' outputs as they are, bit by bit."""
    c = kv_cases.make(131, [37, 150, 700], N, 2, D, 16, stale=NAN)
    q = _queries(132, c, Hq)
    clean, _ = _run_attend(c, q)
    for node in (0, N - 1):
        hit = q.clone()
        hit[:, node] = value
        got, status = _run_attend(c, hit)
        keep = [n for n in range(N) if n != node]
        assert status == 0 and torch.equal(got[:, keep], clean[:, keep])


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("Hq,N", [(8, 4), (8, 61)])
def test_a_large_unseen_vector_costs_no_precision(Hq, N, what):
    """A node's key or value 2^14 times the others', of up to 2^2: its neighbours are rounded to 2^-34 of it at most, 2^-18, which
    is under an eighth of their own half step 2^-11 of what is 2^-4 or larger, and the others' part in a mean is small."""
    c = kv_cases.make(133, [37, 150], N, 2, 128, 16, stale=NAN)
    q = _queries(134, c, Hq)
    codes = kv4_cases.quantised(c)
    want, bound = _expected(c, q, codes, 128 ** -0.5)
    hit = N - 1
    x = getattr(c, what).clone()
    for b in range(2):
        s = int(c.seq_len[b]) + hit
        x[0, int(c.table[b, s // 16]), s % 16] *= 2.0 ** 14
    got, status = _run_attend(kv_cases.dataclasses.replace(c, **{what: x}), q)
    keep = [n for n in range(N) if n != hit]
    err = np.abs(got.double().numpy() - want)[:, keep]
    assert status == 0 and (err <= 1.125 * bound[:, keep]).all()


@pytest.mark.parametrize("N,lens", [(1, [300]), (1, [6000]), (40, [300]), (40, [6000]), (150, [200])])
def test_nan_counts_whatever_its_weight(N, lens):
    """One element of one token's value that is not finite makes its vector NaN, and with it every row that sees it,
    though its weight is 2^-400 of the others'; whoever joins the parts of a split length."""
    c = kv_cases.make(29, lens, N, 1, 64, 16, tree=False, stale=NAN)
    q = _queries(30, c, 4, 0.5)
    q[..., 0] = 16
    for slot in (10, lens[0] // 2, lens[0] - 1):
        k, v = c.k.clone(), c.v.clone()
        k[..., 0] = torch.where(torch.isfinite(k[..., 0]), torch.zeros(()).to(c.dtype), k[..., 0])
        at = (0, int(c.table[0, slot // 16]), slot % 16)
        k[at][..., 0] = -140.0
        v[at][..., 7] = INF
        got, status = _run_attend(kv_cases.dataclasses.replace(c, k=k, v=v), q)
        assert status == 0 and got.isnan().all()


def test_nodes_that_do_not_exist_give_zeros():
    for N, Hq in ((10, 4), (3, 4)):
        c = kv_cases.make(31, [40, 8], N, 1, 64, 16, counts=[2, 0], stale=NAN)
        got, status = _run_attend(c, _queries(32, c, Hq))
        assert status == 0 and (got[0, 2:] == 0).all() and (got[1] == 0).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("N", [1, 12])
def test_strided_queries_and_outputs(N):
    c = kv_cases.make(33, [66, 20], N, 2, 128, 16)
    q = _queries(34, c, 4)
    ref, _ = _run_attend(c, q)
    packed = torch.zeros((2, N, 8, 128), dtype=c.dtype, device="cuda")
    packed[:, :, :4] = q.cuda()
    heads_first = torch.zeros((2, 4, N, 128), dtype=c.dtype, device="cuda")
    status = _status()
    B.spec_tree_kv4_attend(_cache4(c), 0, packed[:, :, :4], heads_first.transpose(1, 2), B.AttendWorkspace(2, N, 4, 2, 128),
                           status, tree=_nodes(c))
    torch.cuda.synchronize()
    assert torch.equal(heads_first.transpose(1, 2).cpu(), ref) and int(status.item()) == 0


@pytest.mark.parametrize("dim", [0, 1, 2])
@pytest.mark.parametrize("N", [2, 12])
def test_broadcast_queries(dim, N):
    """Queries shared by all trees, nodes or heads (stride 0)."""
    c = kv_cases.make(35, [66, 20], N, 2, 128, 16)
    q = _queries(36, c, 4)
    one = q.narrow(dim, 0, 1)
    ref, _ = _run_attend(c, one.expand(q.shape).contiguous())
    status, out = _status(), torch.zeros(q.shape, dtype=c.dtype, device="cuda")
    B.spec_tree_kv4_attend(_cache4(c), 0, one.cuda().expand(q.shape), out, B.AttendWorkspace(2, N, 4, 2, 128), status, tree=_nodes(c))
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref) and int(status.item()) == 0


@pytest.mark.parametrize("N,lens,Hq,D", [(1, [5000], 4, 64), (1, [20000], 8, 128), (61, [6000], 4, 128), (40, [9000], 4, 64),
                                         (2, [3000, 40, 900], 8, 128)])
def test_long_cache_split_and_same_bits(N, lens, Hq, D):
    """Long sequences: their length is split over the card; another run gives the same bits."""
    c = kv_cases.make(37, lens, N, 1, D, 32, tree=N > 1)
    q = _queries(38, c, Hq)
    _check_attend(c, q)
    ws, cache = B.AttendWorkspace(len(lens), N, Hq, 1, D), _cache4(c)
    runs = [_run_attend(c, q, ws=ws, cache=cache)[0] for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_one_workspace_serves_different_calls():
    """Calls of few and many rows, over caches in 4 and in 16 bits, one after the other."""
    a = kv_cases.make(39, [900], 61, 1, 128, 16)
    b = kv_cases.make(40, [20, 2000, 3], 1, 2, 128, 16, tree=False)
    ws = B.AttendWorkspace(3, 61, 8, 1, 128)
    qa, qb = _queries(41, a, 4), _queries(42, b, 4)
    ca, cb, c16 = _cache4(a), _cache4(b), _cache(a)
    ra, rb = _run_attend(a, qa, cache=ca)[0], _run_attend(b, qb, cache=cb)[0]
    out, r16 = [torch.zeros_like(qa, device="cuda") for _ in range(2)]
    status = _status()
    B.spec_tree_attend(c16, 0, qa.cuda(), r16, B.AttendWorkspace(1, 61, 4, 1, 128), status, tree=_nodes(a))
    for _ in range(2):
        assert torch.equal(_run_attend(a, qa, ws=ws, cache=ca)[0], ra)
        assert torch.equal(_run_attend(b, qb, ws=ws, cache=cb)[0], rb)
        B.spec_tree_attend(c16, 0, qa.cuda(), out, ws, status, tree=_nodes(a))
        assert torch.equal(out, r16)


@pytest.mark.parametrize("N", [1, 30])
def test_attention_on_another_stream_and_in_a_graph(N):
    c = kv_cases.make(43, [333, 64], N, 2, 128, 16)
    q = _queries(44, c, 8)
    ref, _ = _run_attend(c, q)
    cache, qd, ws, status, nodes = _cache4(c), q.cuda(), B.AttendWorkspace(2, N, 8, 2, 128), _status(), _nodes(c)
    out = torch.zeros_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.spec_tree_kv4_attend(cache, 0, qd, out, ws, status, tree=nodes, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        B.spec_tree_kv4_attend(cache, 0, qd, out, ws, status, tree=nodes)
    for lens in ([333, 64], [100, 5]):
        cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c2 = kv_cases.dataclasses.replace(c, seq_len=torch.tensor(lens, dtype=torch.int32))
        assert torch.equal(out.cpu(), _run_attend(c2, q)[0])


@pytest.mark.parametrize("N,Hq,Hkv,D,begin", [(8, 16, 4, 64, 25), (1, 32, 8, 128, 0), (61, 8, 8, 128, 0), (61, 8, 2, 128, 0),
                                              (4, 8, 2, 128, 3), (1, 5, 5, 64, 0)])
def test_ragged_batch_many_times(N, Hq, Hkv, D, begin):
    """Rows that are partly nodes that do not exist, segments of every length: a hundred launches of a ragged batch all
    end, in time and with the same bits."""
    rng = np.random.RandomState(1)
    lens = rng.randint(1, 900, 40).tolist()
    counts = [begin + int(rng.randint(0, N + 1)) for _ in lens]
    c = kv_cases.make(45, lens, N, Hkv, D, 32, begin=begin, counts=counts, stale=NAN, tree=N > 1)
    q = _queries(46, c, Hq)
    cache, qd, ws, status, nodes = _cache4(c), q.cuda(), B.AttendWorkspace(40, N, Hq, Hkv, D), _status(), _nodes(c)
    outs = [torch.zeros_like(qd) for _ in range(4)]
    for rep in range(25):
        for out in outs:
            B.spec_tree_kv4_attend(cache, 0, qd, out, ws, status, tree=nodes, node_begin=begin)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(torch.equal(outs[0], o) for o in outs)
    _check_attend(c, q)


@pytest.mark.parametrize("N", [1, 20])
def test_pages_past_32_bit_offsets(N):
    """Pools of more than 2^32 bytes of codes: the pages used lie at their end."""
    page, Hkv, D = 64, 4, 128
    pages = (1 << 33) // (page * Hkv * D) + 40
    c = kv_cases.make(47, [150, 70], N, Hkv, D, page)
    k4, v4, sc = kv4_cases.quantised(c)[:3]
    used = c.k.shape[1]
    k = torch.empty((1, pages, page, Hkv, D // 2), dtype=torch.uint8, device="cuda")
    v, scale = torch.empty_like(k), torch.empty((1, pages, Hkv, page, 4), dtype=c.dtype, device="cuda")
    k[:, pages - used:], v[:, pages - used:], scale[:, pages - used:] = k4.cuda(), v4.cuda(), sc.cuda()
    table = torch.where(c.table >= 0, c.table + (pages - used), c.table).to(torch.int32)
    q = _queries(48, c, 8)
    ref, _ = _run_attend(c, q)
    far = B.KVCache4(k, v, scale, table.cuda(), c.seq_len.cuda())
    got, status = _run_attend(c, q, cache=far)
    assert status == 0 and torch.equal(got, ref)
    # append, read and commit there
    x = torch.randn((2, N, Hkv, D), generator=torch.Generator().manual_seed(0)).to(c.dtype).cuda()
    kr, vr, status = torch.zeros_like(x), torch.zeros_like(x), _status()
    B.spec_tree_kv4_append(far, 0, x, x, -x, torch.zeros_like(x), None, status)
    B.spec_tree_kv4_read(far, 0, kr, vr, status, first=c.seq_len.cuda())
    near = _cache4(c)
    B.spec_tree_kv4_append(near, 0, x, x, -x, torch.zeros_like(x), None, status)
    for cache in (far, near):
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        B.spec_tree_kv4_commit(cache, torch.tensor([N // 7, 0], dtype=torch.int32, device="cuda"),
                               torch.tensor([[3, 5, 9], [0, 0, 0]], dtype=torch.int32, device="cuda"), new, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and float((kr - x).abs().max()) < 0.4
    assert torch.equal(far.k[:, pages - used:], near.k) and torch.equal(far.scale[:, pages - used:], near.scale)


@pytest.mark.parametrize("N", [1, 4, 9])
def test_missing_pages_are_reported(N):
    """An entry outside the pool, and a table that ends early: a status bit, zeros in place of the tokens."""
    c = kv_cases.make(49, [100], N, 1, 64, 16)
    q = _queries(50, c, 2)
    for value in (-1, c.k.shape[1], 1 << 30):
        table = c.table.clone()
        table[0, 2] = value
        got, status = _run_attend(kv_cases.dataclasses.replace(c, table=table), q)
        assert status == B.S_PAGES and torch.isfinite(got.float()).all()
        zeroed = kv_cases.dataclasses.replace(c, k=c.k.clone(), v=c.v.clone())
        zeroed.k[0, int(c.table[0, 2])] = 0
        zeroed.v[0, int(c.table[0, 2])] = 0
        assert torch.equal(got, _run_attend(zeroed, q)[0])
    short = kv_cases.dataclasses.replace(c, table=c.table[:, :3].contiguous())
    got, status = _run_attend(short, q)
    assert status == B.S_PAGES and (got == 0).all()


@pytest.mark.parametrize("N", [6, 20])
def test_bad_parents_and_lengths_are_reported(N):
    c = kv_cases.make(51, [30, 30], N, 1, 64, 16)
    q = _queries(52, c, 2)
    parent = c.parent.clone()
    for up in (5, 3):
        parent[0, 3] = up
        assert _run_attend(kv_cases.dataclasses.replace(c, parent=parent), q)[1] == B.S_NODES
    got, status = _run_attend(kv_cases.dataclasses.replace(c, seq_len=torch.tensor([-4, 30], dtype=torch.int32)), q)
    assert status == B.S_NODES and (got[0] == 0).all()


@pytest.mark.parametrize("Hq,Hkv,N", [(3, 1, 50), (128, 1, 3), (128, 1, 1), (64, 1, 9), (48, 16, 7), (48, 16, 1), (100, 1, 4),
                                      (6, 6, 150), (16, 16, 16)])
def test_group_sizes(Hq, Hkv, N):
    c = kv_cases.make(149, [60, 140], N, Hkv, 64, 16, counts=[N, max(1, N - 2)], stale=NAN)
    _check_attend(c, _queries(151, c, Hq))


def test_chunk_of_a_group_that_does_not_divide_128():
    c = kv_cases.make(152, [75, 300], 90, 1, 128, 32, tree=False, stale=NAN)
    _check_attend(c, _queries(153, c, 7))


@pytest.mark.parametrize("Hq,N", [(4, 3), (4, 40)])
def test_f16_vectors_up_to_the_largest_number(Hq, N):
    c = kv_cases.make(154, [50, 200], N, 2, 64, 16, "f16", stale=NAN)
    v = (c.v.float() * 65504.0).clamp(-65504.0, 65504.0).to(c.dtype)
    k = (c.k.float() * 8192.0).clamp(-65504.0, 65504.0).to(c.dtype)
    c = kv_cases.dataclasses.replace(c, k=torch.where(torch.isfinite(c.k), k, c.k), v=torch.where(torch.isfinite(c.v), v, c.v))
    _check_attend(c, _queries(155, c, Hq, 1.5 / 1024.0), scale=1.0 / 8)


@pytest.mark.parametrize("N", [1, 30])
def test_two_calls_at_once(N):
    """Two streams, a workspace and a status word each: the bits of one call after the other."""
    cases = [kv_cases.make(156 + i, [3000 + 700 * i, 90], N, 2, 128, 16, tree=N > 1) for i in range(2)]
    qs = [_queries(160 + i, c, 8) for i, c in enumerate(cases)]
    want = [_run_attend(c, q)[0] for c, q in zip(cases, qs)]
    caches, nodes, qd = [_cache4(c) for c in cases], [_nodes(c) for c in cases], [q.cuda() for q in qs]
    outs = [torch.full_like(q, NAN) for q in qd]
    wss = [B.AttendWorkspace(2, N, 8, 2, 128) for _ in cases]
    status = [_status() for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                B.spec_tree_kv4_attend(caches[i], 0, qd[i], outs[i], wss[i], status[i], tree=nodes[i], stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert int(status[i].item()) == 0 and torch.equal(outs[i].cpu(), want[i])


# ------------------------------------------------------------------ append ---

def _vectors(seed, shape, dtype):
    """Normal vectors, some of them constant, tiny, far from zero, or with an element that is not finite."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    flat = x.view(-1, shape[-1])
    for i, what in enumerate(("constant", "tiny", "far", "nan", "inf", "wide", "ramp")):
        at = flat[(7 * i + 3) % len(flat)] if len(flat) > 60 else None
        if at is None:
            continue
        if what == "constant":
            at.fill_(1.25)
        elif what == "tiny":
            at.mul_(1e-7)
        elif what == "far":
            at.add_(300.0)
        elif what == "nan":
            at[5] = NAN
        elif what == "inf":
            at[5] = -INF
        elif what == "wide":
            at[:2] = torch.tensor([65504.0, -65504.0]) if dtype == torch.float16 else torch.tensor([3e38, -3e38])
        else:
            at.copy_(torch.arange(shape[-1]) % 31 / 2.0)  # ties
    return x.to(dtype)


def _check_append(seed, lens, N, Hq, Hkv, D, page, dtype="bf16", tree=True, begin=0, counts=None, norm=False, rot=None,
                  interleaved=False, layout="head", layers=1, layer=0, in_place=False, powers=None):
    """Keys, values and queries are to the bit what the append into a 16-bit cache makes of them, quantised."""
    rot = D if rot is None else rot
    c = kv_cases.make(seed, lens, N, Hkv, D, page, dtype, tree=tree, begin=begin, counts=counts, layers=layers)
    q = _queries(seed, c, Hq)
    k, v = (_vectors(seed + i, (len(lens), N, Hkv, D), c.dtype) for i in (1, 2))
    if powers is not None:  # a power of two for each token
        gain = 2.0 ** torch.tensor(powers)[torch.arange(N) % len(powers)].double()[None, :, None, None]
        k, v = ((x.double() * gain).to(c.dtype) for x in (k, v))
    g = torch.Generator().manual_seed(seed)
    qw, kw = [(1 + 0.2 * torch.randn(D, generator=g)).to(c.dtype).cuda() if norm else None for _ in range(2)]
    rope = B.rope_table(max(lens) + begin + N, rot, 10000.0) if rot else None
    before = kv4_cases.quantised(c)
    cache, half = _cache4(c, before, layout), _cache(c)
    status = _status()
    args = dict(tree=_nodes(c), node_begin=begin, q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved)
    q4 = q.cuda()
    out, want_q = (q4 if in_place else torch.full_like(q4, NAN)), torch.full_like(q4, NAN)
    B.spec_tree_kv_append(half, layer, q.cuda(), k.cuda(), v.cuda(), want_q, rope, status, **args)
    B.spec_tree_kv4_append(cache, layer, q4, k.cuda(), v.cuda(), out, rope, status, **args)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(out, want_q)
    wrote = kv_cases.dataclasses.replace(c, k=half.k.cpu(), v=half.v.cpu())
    want = kv4_cases.quantised(wrote)
    for got, w in zip((cache.k.cpu(), cache.v.cpu()), want[:2]):
        assert torch.equal(got, w), int((got != w).sum())
    assert torch.equal(cache.scale.cpu().nan_to_num(nan=-7.0), want[2].nan_to_num(nan=-7.0))
    return c, cache, want


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (128, 16), (64, 0), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, D, rot, interleaved):
    _check_append(60, [0, 33, 100], 21, 4, 2, D, 16, dtype, norm=True, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("kw", [
    dict(lens=[0], N=1, Hq=1, Hkv=1, D=64, page=8, tree=False),
    dict(lens=[700], N=1, Hq=32, Hkv=8, D=128, page=16, tree=False),
    dict(lens=[15, 16, 17], N=40, Hq=5, Hkv=5, D=128, page=16, counts=[40, 17, 0]),
    dict(lens=[9, 300], N=8, Hq=7, Hkv=1, D=64, page=256, begin=17, layout="token"),
    dict(lens=[3], N=90, Hq=4, Hkv=2, D=128, page=64, tree=False, norm=True, layers=3, layer=1),
    dict(lens=[5, 6], N=10, Hq=8, Hkv=2, D=128, page=32, norm=True, in_place=True),
    dict(lens=list(range(40)), N=32, Hq=20, Hkv=3, D=128, page=16, norm=True, rot=0),
    dict(lens=[40, 2], N=64, Hq=2, Hkv=1, D=128, page=16, rot=0, dtype="f16"),
])
def test_append_shapes(kw):
    _check_append(61, **kw)


@pytest.mark.parametrize("dtype,powers", [("bf16", [-136, -131, -127, -124, -100, -64, -60, -57, -30, 30, 57, 62, 64, 100, 121]),
                                          ("f16", [-24, -20, -17, -14, -10, 5, 11, 13])])
def test_append_vectors_of_any_size(dtype, powers):
    """Down to the types' least steps and up to their largest numbers; nothing is turned, which would round."""
    _check_append(62, [9, 300], 45, 4, 2, 128, 16, dtype, rot=0, powers=powers)


def test_append_many_vectors_of_many_ranges():
    """Quotients are those of a division, whatever the step: 100000 vectors."""
    _check_append(63, [0] * 20, 250, 1, 10, 64, 16, "bf16", rot=0, powers=[0])


def test_append_reports_what_it_cannot_place():
    c = kv_cases.make(63, [30], 4, 1, 64, 16, tree=False)
    x = torch.randn((1, 4, 1, 64), generator=torch.Generator().manual_seed(0)).to(c.dtype).cuda()
    codes = kv4_cases.quantised(c)

    def call(table=None, lens=None, rope_rows=40):
        cc = kv_cases.dataclasses.replace(c, table=c.table if table is None else table, seq_len=c.seq_len if lens is None else lens)
        cache, status, out = _cache4(cc, codes), _status(), torch.full_like(x, NAN)
        B.spec_tree_kv4_append(cache, 0, x, x, x, out, B.rope_table(rope_rows, 64), status, tree=_nodes(cc))
        torch.cuda.synchronize()
        return int(status.item()), cache, out.cpu()

    bad = c.table.clone()
    bad[0, 2] = 1 << 29
    status, cache, out = call(table=bad)   # slots 32, 33 have no page; 30, 31 do
    assert status == B.S_PAGES and torch.isfinite(out.float()).all()
    first, k = int(c.table[0, 1]), cache.k.cpu()
    assert not torch.equal(k[0, first, 14:], codes[0][0, first, 14:]) and torch.equal(k[0, first, :14], codes[0][0, first, :14])
    rest = torch.arange(k.shape[1]) != first
    assert torch.equal(k[:, rest], codes[0][:, rest]) and torch.equal(cache.scale.cpu()[:, rest], codes[2][:, rest])
    assert call(rope_rows=32)[0] == B.S_NODES
    status, cache, out = call(lens=torch.tensor([-3], dtype=torch.int32))
    assert status == B.S_NODES and torch.equal(cache.k.cpu(), codes[0]) and (out == 0).all()


# -------------------------------------------------------------------- read ---

@pytest.mark.parametrize("dtype,D,page,layout,Hkv", [("bf16", 128, 16, "head", 2), ("f16", 64, 8, "token", 3), ("bf16", 64, 64, "head", 1)])
def test_read(dtype, D, page, layout, Hkv):
    """Values z + s n, rounded once: half a step; zeros where nothing is asked for; what is NaN stays so."""
    c = kv_cases.make(70, [40, 3, 100], 1, Hkv, D, page, dtype, tree=False, layers=2)
    c.k[1, int(c.table[0, 0]), 3, 0, 5] = INF
    codes = kv4_cases.quantised(c)
    cache, n = _cache4(c, codes, layout), 30
    first, counts = torch.tensor([2, 0, 71], dtype=torch.int32), torch.tensor([30, 4, 12], dtype=torch.int32)
    packed = torch.full((3, n, 2 * Hkv, D), NAN, dtype=c.dtype, device="cuda")
    k, v, status = packed[:, :, :Hkv], packed[:, :, Hkv:], _status()
    B.spec_tree_kv4_read(cache, 1, k, v, status, first=first.cuda(), counts=counts.cuda())
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for got, pool in ((k, codes[3]), (v, codes[4])):
        want = np.zeros((3, n, Hkv, D))
        for b in range(3):
            for i in range(int(counts[b])):
                s = int(first[b]) + i
                want[b, i] = pool[1, int(c.table[b, s // page]), s % page]
        got = got.double().cpu().numpy()
        fine = np.isfinite(want)
        assert np.array_equal(fine, np.isfinite(got)) and (~fine).sum() == (D if pool is codes[3] else 0)
        h = kv_cases.half_step(c.dtype)
        assert (np.abs(got - want)[fine] <= (h * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -25 * np.abs(want).max(-1, keepdims=True))[fine]).all()


def test_read_all_and_what_has_no_page():
    c = kv_cases.make(71, [20, 5], 1, 1, 64, 16, tree=False)
    codes = kv4_cases.quantised(c)
    cache, status = _cache4(c, codes), _status()
    k, v = (torch.full((2, 32, 1, 64), NAN, dtype=c.dtype, device="cuda") for _ in range(2))
    B.spec_tree_kv4_read(cache, 0, k, v, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_PAGES          # the second sequence has one page
    assert (k[1, 16:] == 0).all() and (v[1, 16:] == 0).all() and torch.isfinite(k).all()
    table = c.table[0, :2].long()
    want = torch.from_numpy(codes[3][0])[table].reshape(32, 1, 64).to(c.dtype)
    assert torch.equal(k[0].cpu(), want)
    status.zero_()
    B.spec_tree_kv4_read(cache, 0, k, v, status, first=torch.tensor([-3, 1], dtype=torch.int32, device="cuda"),
                         counts=torch.tensor([5, 9], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_PAGES and (k[0, :3] == 0).all() and torch.equal(k[0, 3:5].cpu(), want[:2]) and (k[1, 9:] == 0).all()


# ------------------------------------------------------------------ commit ---

@pytest.mark.parametrize("dtype,D,page,layout,layers", [("bf16", 128, 16, "token", 3), ("f16", 64, 8, "head", 1),
                                                        ("bf16", 64, 64, "head", 2)])
def test_commit(dtype, D, page, layout, layers):
    lens = [0, 15, 40, 7, 100]
    c = kv_cases.make(80, lens, 61, 2, D, page, dtype, layers=layers)
    nodes = [[3, 9, 20, 33, 41, 50, 55, 60], [1, 2, 3, 4, 5, 6, 7, 8], [8] + [-1] * 7, [-1] * 8, [2, 3, 5, 8, 13, 21, -1, -1]]
    accept = [8, 8, 1, 0, 6]
    out_node = torch.tensor([n + [-1] for n in nodes], dtype=torch.int32)
    codes = kv4_cases.quantised(c)
    cache, status = _cache4(c, codes, layout), _status()
    new = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    B.spec_tree_kv4_commit(cache, torch.tensor(accept, dtype=torch.int32, device="cuda"), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    k, v, want = O.commit(codes[0].numpy(), codes[1].numpy(), c.table.numpy(), lens, accept, out_node.numpy())
    four = np.swapaxes(codes[2].double().numpy(), 2, 3)
    four, _, _ = O.commit(four, four, c.table.numpy(), lens, accept, out_node.numpy())
    assert int(status.item()) == 0 and new.tolist() == want.tolist()
    assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)
    assert np.array_equal(cache.scale.double().cpu().numpy(), np.swapaxes(four, 2, 3))


def test_commit_long_path():
    """A path of 255 nodes (more than one batch of the kernel's loads), each step's source another's destination."""
    c = kv_cases.make(81, [11], 300, 1, 64, 16, tree=False)
    ids = list(range(3, 258))
    codes = kv4_cases.quantised(c)
    cache, status, new = _cache4(c, codes), _status(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out_node = torch.tensor([ids + [-1]], dtype=torch.int32)
    B.spec_tree_kv4_commit(cache, torch.tensor([255], dtype=torch.int32, device="cuda"), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    k, v, want = O.commit(codes[0].numpy(), codes[1].numpy(), c.table.numpy(), [11], [255], out_node.numpy())
    assert int(status.item()) == 0 and new.tolist() == want.tolist()
    assert np.array_equal(cache.k.cpu().numpy(), k) and np.array_equal(cache.v.cpu().numpy(), v)


def test_commit_leaves_bad_paths_alone():
    c = kv_cases.make(82, [20, 20, 20, -1, 20], 12, 1, 64, 16, tree=False)
    out_node = torch.tensor([[2, 1, -1], [1, 2, -1], [1, 2, 3], [1, 2, -1], [4, -2, 5]], dtype=torch.int32)
    acc = torch.tensor([2, 2, 4, 2, 2], dtype=torch.int32)
    codes = kv4_cases.quantised(c)
    cache, status, new = _cache4(c, codes), _status(), torch.zeros(5, dtype=torch.int32, device="cuda")
    B.spec_tree_kv4_commit(cache, acc.cuda(), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_NODES and new.tolist() == [20, 23, 20, -1, 20]
    assert torch.equal(cache.k.cpu(), codes[0]) and torch.equal(cache.scale.cpu().nan_to_num(), codes[2].nan_to_num())


# ------------------------------------------------------------------- pages ---

def _same(pool, want, stack_too=True):
    held = pool.held.tolist()
    assert held == [len(r) for r in want.rows] and int(pool.n_free[0]) == len(want.stack)
    for row, h, r in zip(pool.page_table.tolist(), held, want.rows):
        assert row[:h] == r and all(x == -1 for x in row[h:])
    assert pool.free.tolist()[:len(want.stack)] == want.stack


@pytest.mark.parametrize("B_,page,seed", [(1, 8, 0), (7, 16, 1), (64, 16, 2), (600, 32, 3), (1500, 8, 4)])
def test_pages_of_a_running_server(B_, page, seed):
    """Steps of a batch whose sequences grow, shrink and end, with the pages running out now and then."""
    rng = np.random.RandomState(seed)
    width = 12
    n_pages = max(3, B_ * width // 3)
    pool = B.PagePool(n_pages, page, B_, width)
    want = O4.Pages(B_, n_pages, page, width, range(n_pages - 1, -1, -1))
    up = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    ran_out = 0
    for step in range(6):
        count = int(rng.choice([1, 5, 61]))
        lens = rng.randint(0, width * page - (0 if step == 3 else min(61, width * page - 1)), B_)
        if B_ > 1 and step == 2:
            lens[rng.randint(B_)] = -1
        n_nodes = rng.randint(-1, count + 3, B_) if step % 2 else None
        status, slots = _status(), torch.full((B_, count), -9, dtype=torch.int64, device="cuda")
        B.spec_tree_kv_reserve(pool, up(lens), count, status, n_nodes=None if n_nodes is None else up(n_nodes),
                               slots=slots if step != 4 else None)
        torch.cuda.synchronize()
        expect, short = want.reserve(lens.tolist(), count, None if n_nodes is None else n_nodes.tolist())
        assert int(status.item()) == (B.S_PAGES if short else 0) | (B.S_NODES if (lens < 0).any() else 0)
        if step != 4:
            assert slots.tolist() == expect
        _same(pool, want)
        ran_out += short
        keep = np.where(rng.rand(B_) < 0.4, 0, rng.randint(0, width * page, B_))
        status.zero_()
        if B_ > 1 and step == 1:
            keep[0] = -5
        B.spec_tree_kv_release(pool, up(keep), status)
        torch.cuda.synchronize()
        want.release(keep.tolist())
        assert int(status.item()) == (B.S_NODES if (keep < 0).any() else 0)
        _same(pool, want)
        assert not pool.scratch.any()
    assert ran_out or B_ == 1
    B.spec_tree_kv_release(pool, up(np.zeros(B_)), status)
    torch.cuda.synchronize()
    assert int(pool.n_free[0]) == n_pages and sorted(pool.free.tolist()) == list(range(n_pages))


def test_long_prompts_are_given_their_pages():
    """Rows of thousands of pages, a table that is wider than what a call may use."""
    big = torch.full((3, 9000), -1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.randperm(20000, generator=torch.Generator().manual_seed(0)).to(**i32)
    pool = B.PagePool(20000, 16, 3, 8192, big[:, :8192], torch.zeros(3, **i32), free, torch.full((1,), 20000, **i32))
    status = _status()
    order = free.tolist()[::-1]
    B.spec_tree_kv_reserve(pool, torch.tensor([131071, 131072, 70000], **i32), 1, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_PAGES and pool.held.tolist() == [8192, 0, 4376]
    assert big[0].tolist() == order[:8192] + [-1] * 808 and big[2, :4376].tolist() == order[8192:8192 + 4376]
    B.spec_tree_kv_release(pool, torch.zeros(3, **i32), status)
    torch.cuda.synchronize()
    assert (big == -1).all() and pool.free.tolist() == order[::-1]


def test_a_pool_that_would_overflow_is_left_alone():
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = B.PagePool(4, 16, 1, 4, torch.tensor([[0, 1, 2, 3]], **i32), torch.tensor([4], **i32),
                      torch.tensor([3, 2, -1, -1], **i32), torch.tensor([2], **i32))  # pages 2 and 3 are in two places
    status = _status()
    B.spec_tree_kv_release(pool, torch.tensor([16], **i32), status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_PAGES and pool.held.tolist() == [4] and pool.page_table.tolist() == [[0, 1, 2, 3]]
    assert pool.free.tolist() == [3, 2, -1, -1] and int(pool.n_free[0]) == 2


# ------------------------------------------------------------- all together ---

def test_a_step_in_a_graph():
    """Pages reserved, a tree appended, attended to and committed, unneeded pages given back: captured once and replayed
    from other lengths, it does what the calls do one by one."""
    Bn, N, Hq, Hkv, D, page, width = 3, 21, 4, 2, 64, 16, 12
    rng = np.random.RandomState(0)
    trees = [kv_cases.random_tree(rng, N) for _ in range(Bn)]
    nodes = B.NodeArrays(torch.from_numpy(np.stack([t[0] for t in trees])).cuda(),
                         torch.from_numpy(np.stack([t[1] for t in trees])).cuda())
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    x = torch.randn((Bn, N, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    prompt = torch.randn((Bn, 90, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    rope = B.rope_table(256, D)
    path = torch.full((Bn, 9), -1, dtype=torch.int32)
    accept = []
    for b, (parent, depth) in enumerate(trees):
        chain, at = [], int(np.argmax(depth))
        while at > 0:
            chain.append(at)
            at = int(parent[at])
        path[b, :len(chain)] = torch.tensor(chain[::-1])
        accept.append(len(chain))
    path, accept = path.cuda(), torch.tensor(accept, **i32)

    def fresh():
        pool = B.PagePool(Bn * width, page, Bn, width)
        lens = torch.zeros(Bn, **i32)
        cache = B.KVCache4.zeros(1, Bn * width, page, Hkv, D, pool.page_table, lens)
        s = dict(pool=pool, cache=cache, lens=lens, status=_status(), out=torch.zeros((Bn, N, Hq, D), dtype=torch.bfloat16, device="cuda"),
                 new=torch.zeros(Bn, **i32), ws=B.AttendWorkspace(Bn, 90, Hq, Hkv, D),
                 q=torch.zeros((Bn, N, Hq, D), dtype=torch.bfloat16, device="cuda"))
        B.spec_tree_kv_reserve(pool, lens, 90, s["status"])
        p = prompt.clone()
        B.spec_tree_kv4_append(cache, 0, p[:, :, :Hq], p[:, :, Hq:Hq + Hkv], p[:, :, Hq + Hkv:], p[:, :, :Hq], rope, s["status"])
        B.spec_tree_kv_release(pool, torch.tensor([90, 33, 64], **i32), s["status"])
        lens.copy_(torch.tensor([90, 33, 64]))
        return s

    def step(s):
        B.spec_tree_kv_reserve(s["pool"], s["lens"], N, s["status"])
        B.spec_tree_kv4_append(s["cache"], 0, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], s["q"], rope, s["status"], tree=nodes)
        B.spec_tree_kv4_attend(s["cache"], 0, s["q"], s["out"], s["ws"], s["status"], tree=nodes)
        B.spec_tree_kv4_commit(s["cache"], accept, path, s["new"], s["status"])
        B.spec_tree_kv_release(s["pool"], s["new"], s["status"])
        s["lens"].copy_(s["new"])

    plain, graphed = fresh(), fresh()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(graphed)
    for _ in range(4):
        step(plain)
        graph.replay()
        torch.cuda.synchronize()
        assert int(plain["status"].item()) == int(graphed["status"].item()) == 0
        for name in ("out", "lens"):
            assert torch.equal(plain[name], graphed[name])
        assert torch.equal(plain["pool"].page_table, graphed["pool"].page_table)
        assert torch.equal(plain["cache"].k, graphed["cache"].k) and torch.equal(plain["cache"].scale, graphed["cache"].scale)
        assert (plain["pool"].held == (plain["lens"] + page - 1) // page).all()


# ------------------------------------------------------------- all together ---

def test_a_loop_of_drafting_verification_and_commit():
    """Rounds over caches in 4 bits, with pages from a pool: the first layer's entries of the committed tokens are those of a
    plain pass over them, up to half a step of each side's codes, two roundings to bf16 in the layer and one as they are read
    back (half a step, 2^-8, each); every page belongs to one sequence or is free."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tree_decode
    target, tokens, accepted = tree_decode.decode(B=3, rounds=8, bits=4)
    assert max(map(max, accepted)) > 0
    lengths = target.cache.seq_len.tolist()
    assert lengths == [len(t) - 1 for t in tokens]
    pool, free = target.pool, int(target.pool.n_free.item())
    assert pool.held.tolist() == [-(-n // pool.page_size) for n in lengths]
    mine = [target.pool.page_table[b, :n].tolist() for b, n in enumerate(pool.held.tolist())]
    assert sorted(sum(mine, []) + pool.free[:free].tolist()) == list(range(pool.n_pages))
    status = _status()

    def entries(model, b, n):
        out = [torch.empty((3, max(lengths), 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        counts = torch.zeros(3, dtype=torch.int32, device="cuda")
        counts[b] = n  # the others may be shorter, without pages so far
        B.spec_tree_kv4_read(model.cache, 0, *out, status, counts=counts)
        slots = torch.arange(n, device="cuda")
        pages = model.cache.page_table[b].long()[slots // pool.page_size]
        steps = model.cache.scale[0, pages, :, slots % pool.page_size].double()
        return [(x[b, :n].double(), steps[..., 2 * i, None]) for i, x in enumerate(out)]

    for b, row in enumerate(tokens):
        plain = tree_decode.Model(0, 3, target.rope.shape[0], 4096, 2, max_nodes=256, bits=4)
        plain.step(torch.tensor([row[:-1]] * 3, device="cuda"), status)
        for (a, sa), (c, sc) in zip(entries(target, b, lengths[b]), entries(plain, b, lengths[b])):
            largest = torch.maximum(a.abs(), c.abs()).amax(-1, keepdim=True)
            assert bool(((a - c).abs() <= (sa + sc) / 2 + 6 * 2.0 ** -8 * largest).all())
    assert int(status.item()) == 0
