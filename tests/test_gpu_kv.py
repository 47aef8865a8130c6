"""The paged key-value cache on the GPU against the float64 oracle: append, tree attention, commit."""
import numpy as np
import pytest
import torch

import kv_cases
from dynamic_tree_speculative_gb300 import binding as B
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu


def _cache(c):
    """The case's cache on the GPU, its strides kept."""
    def there(x):
        if x.is_contiguous():
            return x.cuda()
        return x.transpose(2, 3).contiguous().cuda().transpose(2, 3)
    return B.KVCache(there(c.k), there(c.v), c.table.cuda(), c.seq_len.cuda())


def _nodes(c):
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return None if c.parent is None and c.n_nodes is None else B.NodeArrays(up(c.parent), up(c.depth), up(c.n_nodes))


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _queries(seed, c, Hq, gain=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((len(c.counts), c.N, Hq, c.k.shape[4]), generator=g) * gain).to(c.dtype)


def _run_attend(c, q, scale=None, layer=0, ws=None, cache=None):
    cache = cache or _cache(c)
    qd = q.cuda()
    out = torch.full(qd.shape, float("nan"), dtype=c.dtype, device="cuda")
    ws = ws or B.AttendWorkspace(cache.B, c.N, q.shape[2], c.k.shape[3], c.k.shape[4])
    status = _status()
    B.spec_tree_attend(cache, layer, qd, out, ws, status, tree=_nodes(c), node_begin=c.begin, scale=scale)
    torch.cuda.synchronize()
    return out.cpu(), int(status.item())


def _check_attend(c, q, scale=None, layer=0):
    D = c.k.shape[4]
    got, status = _run_attend(c, q, scale, layer)
    k, v = c.pools(layer)
    parents = None if c.parent is None else c.parent.numpy()
    want, mean_abs, score_abs, sum_abs = O.attend(q.double().numpy(), k, v, c.table.numpy(), c.seq_len.numpy(), parents,
                                                  c.counts, c.begin, D ** -0.5 if scale is None else scale)
    tokens = int(c.seq_len.max()) + c.begin + c.N
    bound = kv_cases.attend_bound(c.dtype, want, mean_abs, score_abs, sum_abs, D, tokens)
    err = np.abs(got.double().numpy() - want)
    assert status == 0 and (err <= bound).all(), (status, float(np.nanmax(err / bound)), int((~(err <= bound)).sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[0], [1], [5, 0, 127], [128, 129, 300], [1000, 3]])
def test_one_token(dtype, D, lens):
    c = kv_cases.make(1, lens, 1, 2, D, 16, dtype, tree=False, stale=float("nan"))
    _check_attend(c, _queries(2, c, 8))


@pytest.mark.parametrize("lens", [[0], [3, 64, 130], [70, 515]])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(8, 2, 128, "bf16"), (2, 2, 128, "f16"), (4, 4, 64, "bf16"),
                                            (7, 1, 64, "f16"), (10, 2, 128, "bf16")])
def test_tree(lens, Hq, Hkv, D, dtype):
    c = kv_cases.make(3, lens, 61, Hkv, D, 16, dtype, stale=float("inf"))
    _check_attend(c, _queries(4, c, Hq))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 512])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_pages(page, layout):
    c = kv_cases.make(5, [200, 61, 7], 33, 2, 128, page, layout=layout, stale=float("nan"))
    _check_attend(c, _queries(6, c, 4))


@pytest.mark.parametrize("n", [1, 2, 17, 64, 65, 127, 128, 129, 200])
def test_tree_sizes(n):
    c = kv_cases.make(7, [90, 40], n, 1, 64, 32, tree=True, counts=[n, max(1, n - 5)], stale=float("nan"))
    _check_attend(c, _queries(8, c, 3))


def test_largest_tree():
    c = kv_cases.make(9, [33], 512, 1, 64, 32)
    _check_attend(c, _queries(10, c, 2))


@pytest.mark.parametrize("begin,N", [(1, 8), (9, 8), (25, 8), (130, 6), (0, 1)])
def test_frontier(begin, N):
    """A drafter's frontier: the call's nodes come behind earlier ones, whose entries are in the cache."""
    c = kv_cases.make(11, [100, 31, 0], N, 2, 64, 16, begin=begin, counts=[begin + N, begin + N - 1, begin],
                      stale=float("nan"))
    _check_attend(c, _queries(12, c, 8))


@pytest.mark.parametrize("N,lens,Hq,Hkv", [(40, [0], 4, 1), (130, [77], 4, 2), (300, [10, 500], 2, 1), (600, [0], 1, 1)])
def test_chunk(N, lens, Hq, Hkv):
    c = kv_cases.make(13, lens, N, Hkv, 128, 64, tree=False, stale=float("nan"))
    _check_attend(c, _queries(14, c, Hq))


def test_chain_begin_and_counts():
    c = kv_cases.make(15, [50, 9, 4], 70, 1, 128, 16, tree=False, begin=30, counts=[100, 41, 30], stale=float("nan"))
    _check_attend(c, _queries(16, c, 4))


def test_many_short_sequences():
    rng = np.random.RandomState(0)
    c = kv_cases.make(17, rng.randint(0, 60, 300).tolist(), 1, 1, 64, 8, tree=False, stale=float("nan"))
    _check_attend(c, _queries(18, c, 2))


def test_layers_and_scale():
    c = kv_cases.make(19, [140, 20], 9, 2, 128, 16, layers=3, stale=float("nan"))
    for layer in (0, 2):
        _check_attend(c, _queries(20, c, 4), scale=0.31, layer=layer)
    _check_attend(c, _queries(20, c, 4), scale=0.0)
    _check_attend(c, _queries(20, c, 4), scale=-0.05)


def test_sharp_scores():
    """Scores spread over hundreds: the running maximum moves by more than any threshold, both ways."""
    c = kv_cases.make(21, [700, 260], 12, 1, 128, 16)
    for order in (1, -1):
        k = c.k.clone()
        for b, n in enumerate(c.seq_len.tolist()):
            for s in range(n):
                k[0, int(c.table[b, s // 16]), s % 16] *= (s if order > 0 else n - s) / 40.0
        _check_attend(kv_cases.dataclasses.replace(c, k=k), _queries(22, c, 4))


def test_unseen_nodes_have_no_influence():
    """NaN and infinities in nodes off the path (keys, values): only their descendants feel them."""
    c = kv_cases.make(23, [37, 150], 61, 2, 128, 16, stale=float("nan"))
    q = _queries(24, c, 8)
    clean, _ = _run_attend(c, q)
    for what, value in (("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("k", float("inf"))):
        hit = 20
        x = getattr(c, what).clone()
        for b in range(2):
            s = int(c.seq_len[b]) + hit
            x[0, int(c.table[b, s // 16]), s % 16] = value
        got, status = _run_attend(kv_cases.dataclasses.replace(c, **{what: x}), q)
        assert status == 0
        for b in range(2):
            for n in range(61):
                if hit in O.sees(c.parent[b].numpy(), n):
                    if value != value or what == "v":
                        assert not torch.isfinite(got[b, n]).any(), (what, value, b, n)
                else:
                    assert torch.equal(got[b, n], clean[b, n]), (what, value, b, n)


def test_infinite_values_keep_their_sign_and_place():
    """One element of one seen node's value is infinite: that element of its descendants' outputs is, no other."""
    c = kv_cases.make(25, [130], 20, 1, 64, 16)
    q = _queries(26, c, 2)
    clean, _ = _run_attend(c, q)
    for value in (float("inf"), float("-inf")):
        v, s = c.v.clone(), 130 + 6
        v[0, int(c.table[0, s // 16]), s % 16, 0, 11] = value
        got, _ = _run_attend(kv_cases.dataclasses.replace(c, v=v), q)
        for n in range(20):
            seen = 6 in O.sees(c.parent[0].numpy(), n)
            assert (got[0, n, :, 11] == value).all() if seen else torch.equal(got[0, n], clean[0, n])
            rest = torch.arange(64) != 11
            assert torch.equal(got[0, n][:, rest], clean[0, n][:, rest])


def test_infinite_scores():
    """A token whose score is -inf has no weight; a node that sees nothing else gets zeros."""
    c = kv_cases.make(27, [6], 4, 1, 64, 16, tree=False)
    q = torch.ones((1, 4, 2, 64)).to(c.dtype)
    k = c.k.clone()
    at = lambda s: (0, int(c.table[0, s // 16]), s % 16)  # noqa: E731
    k[at(2)] = float("-inf")
    _check_attend(kv_cases.dataclasses.replace(c, k=k), q)
    for s in range(8):
        k[at(s)] = float("-inf")
    got, _ = _run_attend(kv_cases.dataclasses.replace(c, k=k), q)
    assert (got[0, :2] == 0).all() and torch.isfinite(got[0, 2:].float()).all() and (got[0, 2:] != 0).any()


def test_nodes_that_do_not_exist_give_zeros():
    c = kv_cases.make(29, [40, 8], 10, 1, 64, 16, counts=[4, 0], stale=float("nan"))
    got, status = _run_attend(c, _queries(30, c, 4))
    assert status == 0 and (got[0, 4:] == 0).all() and (got[1] == 0).all() and torch.isfinite(got).all()


def test_strided_queries_and_outputs():
    c = kv_cases.make(31, [66, 20], 12, 2, 128, 16)
    q = _queries(32, c, 4)
    ref, _ = _run_attend(c, q)
    cache = _cache(c)
    packed = torch.zeros((2, 12, 8, 128), dtype=c.dtype, device="cuda")
    packed[:, :, :4] = q.cuda()
    heads_first = torch.zeros((2, 4, 12, 128), dtype=c.dtype, device="cuda")
    status = _status()
    B.spec_tree_attend(cache, 0, packed[:, :, :4], heads_first.transpose(1, 2), B.AttendWorkspace(2, 12, 4, 2, 128), status,
                       tree=_nodes(c))
    torch.cuda.synchronize()
    assert torch.equal(heads_first.transpose(1, 2).cpu(), ref) and int(status.item()) == 0


def test_long_cache_split_and_same_bits():
    """One long sequence: its length is split over the card; a second run gives the same bits."""
    c = kv_cases.make(33, [5000], 1, 1, 64, 32, tree=False)
    q = _queries(34, c, 4)
    _check_attend(c, q)
    ws = B.AttendWorkspace(1, 1, 4, 1, 64)
    runs = [_run_attend(c, q, ws=ws)[0] for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_one_workspace_serves_different_calls():
    a = kv_cases.make(35, [900], 61, 1, 128, 16)
    b = kv_cases.make(36, [20, 2000, 3], 1, 2, 128, 16, tree=False)
    ws = B.AttendWorkspace(3, 61, 8, 1, 128)
    qa, qb = _queries(37, a, 4), _queries(38, b, 4)
    ra, rb = _run_attend(a, qa)[0], _run_attend(b, qb)[0]
    for _ in range(2):
        assert torch.equal(_run_attend(a, qa, ws=ws)[0], ra)
        assert torch.equal(_run_attend(b, qb, ws=ws)[0], rb)


def test_attention_on_another_stream_and_in_a_graph():
    c = kv_cases.make(39, [333, 64], 30, 2, 128, 16)
    q = _queries(40, c, 8)
    ref, _ = _run_attend(c, q)
    cache, qd, ws, status, nodes = _cache(c), q.cuda(), B.AttendWorkspace(2, 30, 8, 2, 128), _status(), _nodes(c)
    out = torch.zeros_like(qd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.spec_tree_attend(cache, 0, qd, out, ws, status, tree=nodes, stream=side)
    side.synchronize()
    assert torch.equal(out.cpu(), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        B.spec_tree_attend(cache, 0, qd, out, ws, status, tree=nodes)
    for lens in ([333, 64], [100, 5]):
        cache.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        c2 = kv_cases.dataclasses.replace(c, seq_len=torch.tensor(lens, dtype=torch.int32))
        assert torch.equal(out.cpu(), _run_attend(c2, q)[0])


@pytest.mark.parametrize("N,Hq,Hkv,D,begin", [(8, 16, 4, 64, 25), (1, 32, 8, 128, 0), (61, 8, 8, 128, 0), (61, 8, 2, 128, 0)])
def test_ragged_batch_many_times(N, Hq, Hkv, D, begin):
    """Warps whose lanes are partly nodes that do not exist, segments of every length: a hundred launches of a
    ragged batch all end, in time and with the same bits."""
    rng = np.random.RandomState(1)
    lens = rng.randint(1, 900, 40).tolist()
    counts = [begin + int(rng.randint(0, N + 1)) for _ in lens]
    c = kv_cases.make(47, lens, N, Hkv, D, 32, begin=begin, counts=counts, stale=float("nan"), tree=N > 1)
    q = _queries(48, c, Hq)
    cache, qd, ws, status, nodes = _cache(c), q.cuda(), B.AttendWorkspace(40, N, Hq, Hkv, D), _status(), _nodes(c)
    outs = [torch.zeros_like(qd) for _ in range(4)]
    for rep in range(25):
        for out in outs:
            B.spec_tree_attend(cache, 0, qd, out, ws, status, tree=nodes, node_begin=begin)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(torch.equal(outs[0], o) for o in outs)
    _check_attend(c, q)


def test_pages_past_32_bit_offsets():
    """A pool of more than 2^32 elements: the pages used lie at its end."""
    page, Hkv, D = 64, 4, 128
    pages = (1 << 32) // (page * Hkv * D) + 40
    c = kv_cases.make(41, [150, 70], 20, Hkv, D, page)
    used = c.k.shape[1]
    k = torch.empty((1, pages, page, Hkv, D), dtype=c.dtype, device="cuda")
    v = torch.empty_like(k)
    k[:, pages - used:], v[:, pages - used:] = c.k.cuda(), c.v.cuda()
    table = torch.where(c.table >= 0, c.table + (pages - used), c.table).to(torch.int32)
    q = _queries(42, c, 8)
    ref, _ = _run_attend(c, q)
    got, status = _run_attend(c, q, cache=B.KVCache(k, v, table.cuda(), c.seq_len.cuda()))
    assert status == 0 and torch.equal(got, ref)


def test_missing_pages_are_reported():
    """An entry outside the pool, and a table that ends early: a status bit, zeros in place of the tokens."""
    c = kv_cases.make(43, [100], 4, 1, 64, 16)
    q = _queries(44, c, 2)
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
    assert _run_attend(short, q)[1] == B.S_PAGES


def test_bad_parents_and_lengths_are_reported():
    c = kv_cases.make(45, [30, 30], 6, 1, 64, 16)
    q = _queries(46, c, 2)
    parent = c.parent.clone()
    parent[0, 3] = 5
    assert _run_attend(kv_cases.dataclasses.replace(c, parent=parent), q)[1] == B.S_NODES
    parent[0, 3] = 3
    assert _run_attend(kv_cases.dataclasses.replace(c, parent=parent), q)[1] == B.S_NODES
    got, status = _run_attend(kv_cases.dataclasses.replace(c, seq_len=torch.tensor([-4, 30], dtype=torch.int32)), q)
    assert status == B.S_NODES and (got[0] == 0).all()


# ------------------------------------------------------------------ append ---

def _check_append(seed, lens, N, Hq, Hkv, D, page, dtype="bf16", tree=True, begin=0, counts=None, norm=False, rot=None,
                  interleaved=False, layout="token", layers=1, layer=0, in_place=False):
    rot = D if rot is None else rot
    c = kv_cases.make(seed, lens, N, Hkv, D, page, dtype, tree=tree, begin=begin, counts=counts, layers=layers, layout=layout)
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((len(lens), N, Hq + 2 * Hkv, D), generator=g).to(c.dtype)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    qw, kw = [(1 + 0.2 * torch.randn(D, generator=g)).to(c.dtype) if norm else None for _ in range(2)]
    rope = B.rope_table(max(lens) + begin + N, rot, 10000.0, "cpu") if rot else None
    cache, packed = _cache(c), qkv.cuda()
    dq, dk, dv = packed[:, :, :Hq], packed[:, :, Hq:Hq + Hkv], packed[:, :, Hq + Hkv:]
    out = dq if in_place else torch.full(q.shape, float("nan"), dtype=c.dtype, device="cuda")
    status = _status()
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    B.spec_tree_kv_append(cache, layer, dq, dk, dv, out, up(rope), status, tree=_nodes(c), node_begin=begin,
                          q_weight=up(qw), k_weight=up(kw), eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    kp, vp = c.pools(layer)
    wq, wk, wv = O.append(f64(q), f64(k), f64(v), kp, vp, c.table.numpy(), c.seq_len.numpy(),
                          None if c.depth is None else c.depth.numpy(), c.counts, begin, f64(rope), rot, interleaved,
                          f64(qw), f64(kw), 1e-5)
    assert int(status.item()) == 0
    assert np.array_equal(f64(cache.v.cpu())[layer], wv)
    # one rounding to dtype; before it the norm (a sum of D squares, a root, two products) and two products
    # and a sum of values of up to the vector's largest, in float32
    for got, want in ((f64(out.cpu()), wq), (f64(cache.k.cpu())[layer], wk)):
        largest = np.abs(want).max(-1, keepdims=True)
        bound = kv_cases.half_step(c.dtype) * np.abs(want) + (D / 2 + 8) * 2.0 ** -23 * largest + 2.0 ** -25
        assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
    for other in range(layers):
        if other != layer:
            assert torch.equal(cache.k[other].cpu(), c.k[other]) and torch.equal(cache.v[other].cpu(), c.v[other])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (128, 16), (64, 0), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(dtype, D, rot, interleaved):
    _check_append(50, [0, 33, 100], 21, 4, 2, D, 16, dtype, norm=True, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("kw", [
    dict(lens=[0], N=1, Hq=1, Hkv=1, D=64, page=8, tree=False),
    dict(lens=[700], N=1, Hq=32, Hkv=8, D=128, page=16, tree=False),
    dict(lens=[15, 16, 17], N=40, Hq=5, Hkv=5, D=128, page=16, counts=[40, 17, 0]),
    dict(lens=[9, 300], N=8, Hq=7, Hkv=1, D=64, page=256, begin=17, layout="head"),
    dict(lens=[3], N=90, Hq=4, Hkv=2, D=128, page=64, tree=False, norm=True, layers=3, layer=1),
    dict(lens=[5, 6], N=10, Hq=8, Hkv=2, D=128, page=32, norm=True, in_place=True),
    dict(lens=list(range(40)), N=32, Hq=20, Hkv=3, D=128, page=16, norm=True),  # a warp takes a node whole
])
def test_append_shapes(kw):
    _check_append(51, **kw)


def test_append_far_positions():
    """Positions past 2^17: the table's rows are taken as they are, no angle is formed in float32."""
    page, far = 512, 150000
    pages = 4
    table = torch.full((1, far // page + 2), -1, dtype=torch.int32)
    table[0, far // page] = 3
    k = torch.zeros((1, pages, page, 1, 64), dtype=torch.bfloat16, device="cuda")
    cache = B.KVCache(k, torch.zeros_like(k), table.cuda(), torch.tensor([far], dtype=torch.int32, device="cuda"))
    x = torch.randn((1, 1, 1, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16)
    rope, status, out = B.rope_table(far + 1, 64, 500000.0), _status(), torch.zeros_like(x, device="cuda")
    B.spec_tree_kv_append(cache, 0, x.cuda(), x.cuda(), x.cuda(), out, rope, status)
    torch.cuda.synchronize()
    a = far * 500000.0 ** (-np.arange(32) / 32)
    want = O.turn(x.double().numpy()[0, 0, 0], None, 0.0, np.concatenate([np.cos(a), np.sin(a)]), 64, False)
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(want).max()
    assert int(status.item()) == 0
    for got in (out[0, 0, 0], cache.k[0, 3, far % page, 0]):
        assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,rows", [(0, 0), (32, 8), (64, 4)])
def test_append_keeps_infinities_where_nothing_turns(rot, rows, interleaved):
    """Without norms the part past rot_dim, and a node outside the table (rows), is a copy: infinities stay, no NaN."""
    c = kv_cases.make(54, [3], 3, 1, 64, 16, tree=False)
    x = torch.randn((1, 3, 1, 64), generator=torch.Generator().manual_seed(1)).to(c.dtype)
    x[0, 1:, 0, 40], x[0, 1:, 0, 51] = float("inf"), float("-inf")
    cache, status, out = _cache(c), _status(), torch.zeros_like(x, device="cuda")
    B.spec_tree_kv_append(cache, 0, x.cuda(), x.cuda(), x.cuda(), out, B.rope_table(rows, rot) if rot else None, status,
                          tree=_nodes(c), interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(status.item()) == (B.S_NODES if rot == 64 else 0)
    slots = c.table[0, 0].item(), slice(3, 6)
    start = rot if rot < 64 else 0       # nodes 1 and 2 lie at positions 4 and 5, past a table of 4 rows
    for got in (out.cpu()[0, 1:], cache.k.cpu()[0][slots][1:]):
        assert torch.equal(got[..., start:], x[0, 1:, :, start:]) and not got.isnan().any()


def test_append_reports_what_it_cannot_place():
    c = kv_cases.make(53, [30], 4, 1, 64, 16, tree=False)
    x = torch.randn((1, 4, 1, 64)).to(c.dtype).cuda()
    before = c.k.clone()

    def call(table=None, lens=None, rope_rows=40):
        cc = kv_cases.dataclasses.replace(c, table=c.table if table is None else table,
                                          seq_len=c.seq_len if lens is None else lens)
        cache, status, out = _cache(cc), _status(), torch.full_like(x, float("nan"))
        B.spec_tree_kv_append(cache, 0, x, x, x, out, B.rope_table(rope_rows, 64), status, tree=_nodes(cc))
        torch.cuda.synchronize()
        return int(status.item()), cache.k.cpu(), out.cpu()

    bad = c.table.clone()
    bad[0, 2] = 1 << 29
    status, k, out = call(table=bad)       # slots 32, 33 have no page; 30, 31 do
    assert status == B.S_PAGES and torch.isfinite(out.float()).all()
    first = int(c.table[0, 1])
    assert not torch.equal(k[0, first, 14:], before[0, first, 14:]) and torch.equal(k[0, first, :14], before[0, first, :14])
    assert torch.equal(k[0, int(c.table[0, 2])], before[0, int(c.table[0, 2])])
    status, _, out = call(rope_rows=32)    # positions 32, 33 are past the table
    assert status == B.S_NODES and torch.equal(out[0, 2:], x[0, 2:].cpu())
    status, k, out = call(lens=torch.tensor([-3], dtype=torch.int32))
    assert status == B.S_NODES and torch.equal(k, before) and (out == 0).all()


# ------------------------------------------------------------------ commit ---

@pytest.mark.parametrize("dtype,D,page,layout,layers", [("bf16", 128, 16, "token", 3), ("f16", 64, 8, "head", 1),
                                                        ("bf16", 64, 64, "token", 2)])
def test_commit(dtype, D, page, layout, layers):
    lens = [0, 15, 40, 7, 100]
    c = kv_cases.make(60, lens, 61, 2, D, page, dtype, layers=layers, layout=layout)
    nodes = [[3, 9, 20, 33, 41, 50, 55, 60], [1, 2, 3, 4, 5, 6, 7, 8], [8] + [-1] * 7, [-1] * 8, [2, 3, 5, 8, 13, 21, -1, -1]]
    accept = [8, 8, 1, 0, 6]
    out_node = torch.tensor([n + [-1] for n in nodes], dtype=torch.int32)
    acc = torch.tensor(accept, dtype=torch.int32)
    cache, status = _cache(c), _status()
    new = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    B.spec_tree_kv_commit(cache, acc.cuda(), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    k, v, want = O.commit(c.k.double().numpy(), c.v.double().numpy(), c.table.numpy(), lens, accept, out_node.numpy())
    assert int(status.item()) == 0 and new.tolist() == want.tolist()
    assert np.array_equal(cache.k.double().cpu().numpy(), k) and np.array_equal(cache.v.double().cpu().numpy(), v)


def test_commit_long_path():
    """A path of 255 nodes (more than one batch of the kernel's loads), each step's source another's destination."""
    c = kv_cases.make(61, [11], 300, 1, 64, 16, tree=False)
    ids = list(range(3, 258))
    cache, status, new = _cache(c), _status(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out_node = torch.tensor([ids + [-1]], dtype=torch.int32)
    B.spec_tree_kv_commit(cache, torch.tensor([255], dtype=torch.int32, device="cuda"), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    k, v, want = O.commit(c.k.double().numpy(), c.v.double().numpy(), c.table.numpy(), [11], [255], out_node.numpy())
    assert int(status.item()) == 0 and new.tolist() == want.tolist()
    assert np.array_equal(cache.k.double().cpu().numpy(), k) and np.array_equal(cache.v.double().cpu().numpy(), v)


def test_commit_leaves_bad_paths_alone():
    c = kv_cases.make(62, [20, 20, 20, -1, 20], 12, 1, 64, 16, tree=False)
    out_node = torch.tensor([[2, 1, -1], [1, 2, -1], [1, 2, 3], [1, 2, -1], [4, -2, 5]], dtype=torch.int32)
    acc = torch.tensor([2, 2, 4, 2, 2], dtype=torch.int32)
    cache, status, new = _cache(c), _status(), torch.zeros(5, dtype=torch.int32, device="cuda")
    B.spec_tree_kv_commit(cache, acc.cuda(), out_node.cuda(), new, status)
    torch.cuda.synchronize()
    assert int(status.item()) == B.S_NODES and new.tolist() == [20, 23, 20, -1, 20]
    assert torch.equal(cache.k.cpu(), c.k)


# ------------------------------------------------------------- all together ---

def test_committed_cache_equals_a_plain_pass_over_the_tokens():
    """Rounds of drafting, verification and commit leave the keys and values that a plain pass over the same
    tokens makes: up to the roundings of two bf16 layers (four of half a step, 2^-8, each)."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import tree_decode
    target, tokens, accepted = tree_decode.decode(B=3, rounds=8)
    assert max(map(max, accepted)) > 0
    lengths = target.cache.seq_len.tolist()
    assert lengths == [len(t) - 1 for t in tokens]
    status = _status()
    for b, row in enumerate(tokens):
        plain = tree_decode.Model(0, 3, target.rope.shape[0], 4096, 2, max_nodes=256)
        plain.step(torch.tensor([row[:-1]] * 3, device="cuda"), status)
        for mine, theirs in ((target.cache.k, plain.cache.k), (target.cache.v, plain.cache.v)):
            size = mine.shape[2]
            slots = torch.arange(lengths[b], device="cuda")
            a = mine[:, target.cache.page_table[b].long()[slots // size], slots % size].double()
            c = theirs[:, plain.cache.page_table[b].long()[slots // size], slots % size].double()
            off = (a - c).norm(dim=-1) / c.norm(dim=-1)
            assert float(off[0].max()) <= 2 * 2.0 ** -8 and float(off.max()) <= 4 * 2.0 ** -8 * 2, off.amax((1, 2))
    assert int(status.item()) == 0


# --------------------------------------------------------- more shapes of heads ---

@pytest.mark.parametrize("Hq,Hkv,N", [(3, 1, 50), (128, 1, 3), (64, 1, 9), (48, 16, 7), (100, 1, 4), (6, 6, 150)])
def test_group_sizes(Hq, Hkv, N):
    c = kv_cases.make(49, [60, 140], N, Hkv, 64, 16, counts=[N, max(1, N - 2)], stale=float("nan"))
    _check_attend(c, _queries(51, c, Hq))


def test_chunk_of_a_group_that_does_not_divide_128():
    c = kv_cases.make(52, [75, 300], 90, 1, 128, 32, tree=False, stale=float("nan"))
    _check_attend(c, _queries(53, c, 7))


@pytest.mark.parametrize("dim", [0, 1, 2])
def test_broadcast_queries(dim):
    """Queries shared by all trees, nodes or heads (stride 0)."""
    c = kv_cases.make(54, [66, 20], 12, 2, 128, 16)
    q = _queries(55, c, 4)
    q = q.narrow(dim, 0, 1).expand(q.shape)
    ref, _ = _run_attend(c, q.contiguous())
    cache, status = _cache(c), _status()
    out = torch.zeros(q.shape, dtype=c.dtype, device="cuda")
    B.spec_tree_attend(cache, 0, q.narrow(dim, 0, 1).cuda().expand(q.shape), out, B.AttendWorkspace(2, 12, 4, 2, 128), status,
                       tree=_nodes(c))
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref) and int(status.item()) == 0


def test_one_long_tree_in_many_parts():
    """A tree over one long sequence: an item in more parts than are joined at a time."""
    c = kv_cases.make(56, [9000], 40, 1, 64, 64)
    _check_attend(c, _queries(57, c, 4))


def test_items_split_between_ranges():
    """More items than CTAs, of unequal lengths: ranges begin and end inside items; many launches, the same bits."""
    rng = np.random.RandomState(3)
    lens = rng.randint(100, 1500, 60).tolist()
    c = kv_cases.make(58, lens, 33, 4, 64, 64)
    q = _queries(59, c, 8)
    cache, qd, nodes, status, ws = _cache(c), q.cuda(), _nodes(c), _status(), B.AttendWorkspace(60, 33, 8, 4, 64)
    outs = [torch.zeros_like(qd) for _ in range(3)]
    for _ in range(20):
        for out in outs:
            B.spec_tree_attend(cache, 0, qd, out, ws, status, tree=nodes)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and all(torch.equal(outs[0], o) for o in outs)
    sub = [0, 17, 59]  # the oracle is slow: three of the trees
    c3 = kv_cases.dataclasses.replace(c, table=c.table[sub], seq_len=c.seq_len[sub], parent=c.parent[sub], depth=c.depth[sub],
                                      counts=[c.counts[i] for i in sub])
    k, v = c.pools(0)
    want, mean_abs, score_abs, sum_abs = O.attend(q[sub].double().numpy(), k, v, c3.table.numpy(), c3.seq_len.numpy(),
                                                  c3.parent.numpy(), c3.counts, 0, 64 ** -0.5)
    bound = kv_cases.attend_bound(c.dtype, want, mean_abs, score_abs, sum_abs, 64, 1533)
    assert (np.abs(outs[0].cpu()[sub].double().numpy() - want) <= bound).all()


# ------------------------------------------------------- values that are not finite ---

INF, NAN = float("inf"), float("nan")


def _ramp(c, q, at_slot):
    """The case with keys (and the queries) whose first element adds at_slot(b, slot) to every score."""
    D, k = c.k.shape[4], c.k.clone()
    size = c.k.shape[2]
    for b, n in enumerate(c.seq_len.tolist()):
        for s in range(n + min(c.counts[b], c.begin + c.N)):
            k[0, int(c.table[b, s // size]), s % size, :, 0] = at_slot(b, s) * D ** 0.5 / 16
    q = q.clone()
    q[..., 0] = 16
    return kv_cases.dataclasses.replace(c, k=k), q


def _check_marks(c, q, marks, repeats=1):
    """marks: (tree, slot, element, value): that element of that slot's value, all heads. Every node that sees it gets
    the value there (NaN for both infinities), whatever its weight; all else is as without marks, to the bit, every time."""
    size = c.v.shape[2]
    v, felt = c.v.clone(), {}
    for b, s, d, value in marks:
        v[0, int(c.table[b, s // size]), s % size, :, d] = value
    clean, status = _run_attend(c, q)
    assert status == 0 and torch.isfinite(clean.float()).all()
    want = clean.float()
    for b, length in enumerate(c.seq_len.tolist()):
        mine = [(s, d, value) for tree, s, d, value in marks if tree == b]
        for i in range(c.N):
            if c.begin + i >= c.counts[b]:
                continue
            seen = set(O.sees(None if c.parent is None else c.parent[b].numpy(), c.begin + i))
            for s, d, value in mine:
                if s < length or s - length in seen:
                    old = want[b, i, :, d]
                    want[b, i, :, d] = torch.where(torch.isfinite(old), value, old + value)
    marked = kv_cases.dataclasses.replace(c, v=v)
    cache, qd, nodes, status = _cache(marked), q.cuda(), _nodes(c), _status()
    ws = B.AttendWorkspace(cache.B, c.N, q.shape[2], c.k.shape[3], c.k.shape[4])
    outs = [torch.zeros_like(qd) for _ in range(3)]
    for _ in range(repeats):
        for out in outs:
            B.spec_tree_attend(cache, 0, qd, out, ws, status, tree=nodes, node_begin=c.begin)
        torch.cuda.synchronize()
        for out in outs:
            got = out.cpu().float()
            off = ~((got == want) | (got.isnan() & want.isnan()))
            assert not off.any(), (int(off.sum()), off.nonzero()[:4].tolist(), got[off][:4], want[off][:4])
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,tree", [(1, False), (20, True), (70, True), (150, False)])
@pytest.mark.parametrize("light", [-28, -300])
def test_infinite_values_of_light_tokens(dtype, D, N, tree, light):
    """Seen tokens of next to no weight (2^-40, below f16's least; 2^-433, below float32's): their infinities count
    wherever they lie, in tiles that every node sees whole and in others."""
    c = kv_cases.make(70, [300], N, 2, D, 16, dtype, tree=tree, stale=NAN)
    slots = [10, 130, 255, 256, 261, 299]
    c, q = _ramp(c, _queries(71, c, 8, 0.5), lambda b, s: light if s in slots else 0.0)
    _check_marks(c, q, [(0, s, 3 + 2 * i, INF if i % 2 else -INF) for i, s in enumerate(slots)])
    _check_marks(c, q, [(0, 10, 3, INF), (0, 299, 3, -INF), (0, 130, 4, NAN), (0, 10, 5, INF), (0, 256, 5, INF)])


@pytest.mark.parametrize("N,tree", [(20, True), (70, True), (150, False)])
def test_infinite_values_of_light_nodes(N, tree):
    c = kv_cases.make(72, [250, 70], N, 2, 64, 16, tree=tree, counts=[N, N - 3], stale=NAN)
    hit = [3, 9, 12]
    c, q = _ramp(c, _queries(73, c, 8, 0.5), lambda b, s: -300.0 if s - (250, 70)[b] in hit else 0.0)
    _check_marks(c, q, [(b, (250, 70)[b] + n, 5 + n, INF) for b in range(2) for n in hit] + [(0, 40, 6, -INF)])


@pytest.mark.parametrize("first,last", [(0.0, 300.0), (300.0, 0.0)])
@pytest.mark.parametrize("N,tree", [(1, False), (20, True), (70, True)])
def test_infinite_values_before_and_after_the_maximum_moves(first, last, N, tree):
    """Two tiles far apart in score, one CTA: the output is rescaled by zero when the second one comes, or the second
    one's weights are zero."""
    c = kv_cases.make(74, [400], N, 1, 128, 16, tree=tree)
    c, q = _ramp(c, _queries(75, c, 4, 0.5), lambda b, s: first if s < 200 else last)
    _check_marks(c, q, [(0, 20, 3, INF), (0, 390, 5, INF), (0, 20, 7, -INF), (0, 390, 7, INF), (0, 150, 8, -INF)])


def _split(name):
    rng = np.random.RandomState(5)
    if name == "one":        # pieces, joined by the last to come
        return kv_cases.make(76, [5000], 1, 1, 64, 32, tree=False), 4
    if name == "tree":       # pieces, joined by a kernel of its own
        return kv_cases.make(77, [6000], 61, 1, 128, 64), 4
    if name == "ones":       # ranges of single tokens
        return kv_cases.make(78, rng.randint(200, 900, 170).tolist(), 1, 1, 64, 32, tree=False), 4
    if name == "frontiers":  # ranges, the halves taking turns at the tiles
        return kv_cases.make(79, rng.randint(200, 900, 60).tolist(), 33, 4, 64, 64), 8
    return kv_cases.make(80, rng.randint(200, 900, 80).tolist(), 61, 2, 64, 64), 8  # ranges, 244 rows


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("name", ["one", "tree", "ones", "frontiers", "trees"])
def test_infinite_values_in_split_items(name, up):
    """Items in parts whose references lie hundreds of binary orders apart, either way round: whoever joins them, an
    infinity in any part counts, launch after launch."""
    c, Hq = _split(name)
    lens = c.seq_len.tolist()
    c, q = _ramp(c, _queries(81, c, Hq, 0.5), lambda b, s: 1500.0 * (s if up else lens[b] - s) / lens[b])
    marks = []
    for b, n in enumerate(lens):
        if b % 3 == 0:
            marks += [(b, 2, 3, INF), (b, n // 2, 5, -INF), (b, n - 1, 7, NAN), (b, 4, 9, INF), (b, n - 2, 9, -INF),
                      (b, n, 11, INF), (b, n // 3, 13, -INF), (b, 2 * n // 3, 13, -INF)]
        elif b % 3 == 1 and c.N > 12:
            marks += [(b, n + 5, 3, INF), (b, n + 12, 4, -INF)]
    _check_marks(c, q, marks, repeats=8)


@pytest.mark.parametrize("lens,N", [([6], 4), ([300], 1), ([300], 40), ([5000], 1), ([5000], 61)])
def test_infinite_values_where_no_score_is_above_minus_infinity(lens, N):
    c = kv_cases.make(82, lens, N, 1, 64, 16, tree=False)
    c = kv_cases.dataclasses.replace(c, k=torch.full_like(c.k, -INF), v=torch.full_like(c.v, INF))
    got, status = _run_attend(c, torch.ones((1, N, 4, 64)).to(c.dtype))
    assert status == 0 and (got == 0).all()


def test_arguments_on_the_cpu_are_refused():
    """Nothing is launched; the same call with all of them on the GPU is."""
    c = kv_cases.make(83, [30, 12], 6, 2, 64, 16)
    cache, nodes, status, ws = _cache(c), _nodes(c), _status(), B.AttendWorkspace(2, 6, 4, 2, 64)
    q = _queries(84, c, 4)
    k = _queries(85, c, 2)
    rope, path = B.rope_table(64, 64), torch.zeros((2, 9), dtype=torch.int32)
    acc, new = torch.zeros((2, 2), dtype=torch.int32)
    here = dict(q=q.cuda(), k=k.cuda(), v=k.cuda(), q_out=torch.zeros_like(q, device="cuda"), rope=rope, status=status)
    B.spec_tree_kv_append(cache, 0, tree=nodes, **here)
    B.spec_tree_attend(cache, 0, here["q"], here["q_out"], ws, status, tree=nodes)
    B.spec_tree_kv_commit(cache, acc.cuda(), path.cuda(), new.cuda(), status)
    torch.cuda.synchronize()
    before = cache.k.clone(), cache.v.clone()
    for name in here:
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_kv_append(cache, 0, tree=nodes, **dict(here, **{name: here[name].cpu()}))
    for qq, out, st in ((q, here["q_out"], status), (here["q"], q, status), (here["q"], here["q_out"], status.cpu())):
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_attend(cache, 0, qq, out, ws, st, tree=nodes)
    cpu = B.NodeArrays(c.parent, c.depth, c.n_nodes)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_attend(cache, 0, here["q"], here["q_out"], ws, status, tree=cpu)
    with pytest.raises(B.SpecTreeError):
        B.KVCache(cache.k, cache.v, c.table, cache.seq_len)
    with pytest.raises(B.SpecTreeError):
        cache.set_lengths(c.seq_len)
    for bad in ((acc, path.cuda(), new.cuda()), (acc.cuda(), path, new.cuda()), (acc.cuda(), path.cuda(), new)):
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_kv_commit(cache, *bad, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
