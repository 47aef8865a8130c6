"""Key-value cache entry points: refusals before any launch, structures, the oracle (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import kv_cases
from oracle import kv_oracle as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def B():
    from dynamic_tree_speculative_gb300 import binding
    return binding


def _kv(B, **kw):
    c = B.c_kv(256, 256, 256, 256, 0, 2048, 128, 128, B.BF16, 1, 4, 16, 1, 128, 8, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _append(B, kv, trees=1, layer=0, nodes=None, hq=4, q=None, rope=256, rows=100, rot=128, qw=None, eps=1e-6):
    h = B.c_heads(256, 512, 512, 128)
    n = nodes or B.c_nodes(None, None, None, 0, 0, 1)
    r = ctypes.byref
    return B._lib.spec_tree_kv_append(trees, r(kv), layer, r(n), hq, r(q or h), r(h), r(h), r(h), VP(rope), rows, rot,
                                      0, VP(qw), None, eps, None, None)


def _attend(B, kv, trees=1, layer=0, nodes=None, hq=4, q=None, out=None, scale=0.1, ws=256, ws_bytes=1 << 40):
    h = B.c_heads(256, 512, 512, 128)
    n = nodes or B.c_nodes(None, None, None, 0, 0, 1)
    r = ctypes.byref
    return B._lib.spec_tree_attend(trees, r(kv), layer, r(n), hq, r(q or h), r(out or B.c_heads(4096, 512, 512, 128)),
                                   scale, VP(ws), ws_bytes, None, None)


def _commit(B, kv, trees=1, stride=9, acc=256, node=256, new=512):
    return B._lib.spec_tree_kv_commit(trees, ctypes.byref(kv), VP(acc), VP(node), stride, VP(new), None, None)


# trees = 0: the checks alone run, no launch follows
def test_accepted_arguments(B):
    kv = _kv(B)
    assert _append(B, kv, trees=0) == B.OK and _attend(B, kv, trees=0) == B.OK and _commit(B, kv, trees=0) == B.OK
    assert _append(B, _kv(B, dtype=B.F16, head_dim=64), trees=0, rot=32) == B.OK
    assert _append(B, kv, trees=0, rope=None, rows=0, rot=0) == B.OK


@pytest.mark.parametrize("field,value,rc", [
    ("dtype", 1, "E_LAYOUT"), ("dtype", 7, "E_LAYOUT"), ("head_dim", 96, "E_PARAM"), ("head_dim", 256, "E_PARAM"),
    ("page_size", 0, "E_PARAM"), ("page_size", 4, "E_PARAM"), ("page_size", 24, "E_PARAM"),
    ("page_size", 1 << 17, "E_PARAM"), ("n_pages", 0, "E_PARAM"), ("n_layers", 0, "E_PARAM"),
    ("n_kv_heads", 0, "E_PARAM"), ("max_pages", 0, "E_PARAM"), ("max_pages", 9, "E_PARAM"),
    ("k", 264, "E_LAYOUT"), ("v", 264, "E_LAYOUT"), ("k", None, "E_PARAM"), ("page_table", None, "E_PARAM"),
    ("seq_len", None, "E_PARAM"), ("token_stride", 130, "E_LAYOUT"), ("head_stride", -128, "E_LAYOUT"),
    ("page_stride", 2052, "E_LAYOUT"),
])
def test_bad_caches(B, field, value, rc):
    kv = _kv(B, **{field: value})
    want = getattr(B, rc)
    assert _append(B, kv, trees=0) == want and _attend(B, kv, trees=0) == want and _commit(B, kv, trees=0) == want


def test_bad_calls(B):
    kv, N = _kv(B), B.c_nodes
    for call in (_append, _attend):
        assert call(B, kv, trees=-1) == B.E_PARAM and call(B, kv, trees=65536) == B.E_PARAM
        assert call(B, kv, trees=0, layer=1) == B.E_PARAM and call(B, kv, trees=0, layer=-1) == B.E_PARAM
        assert call(B, kv, trees=0, nodes=N(None, None, None, 0, 0, 0)) == B.E_PARAM       # no node
        assert call(B, kv, trees=0, nodes=N(None, None, None, 0, -1, 1)) == B.E_PARAM
        assert call(B, kv, trees=0, nodes=N(None, 256, None, 0, 0, 1)) == B.E_PARAM        # depths without parents
        assert call(B, kv, trees=0, nodes=N(None, None, None, 0, 0, (1 << 20) + 1)) == B.E_PARAM
        assert call(B, kv, trees=0, nodes=N(256, 256, None, 10, 3, 8)) == B.E_PARAM        # past the stride
        assert call(B, kv, trees=0, nodes=N(256, 256, None, 1000, 3, 510)) == B.E_PARAM    # past 512 nodes
        assert call(B, kv, trees=0, nodes=N(256, 256, None, 512, 0, 512)) == B.OK
        assert call(B, kv, trees=0, q=B.c_heads(264, 512, 512, 128)) == B.E_LAYOUT
        assert call(B, kv, trees=0, q=B.c_heads(256, 512, 516, 128)) == B.E_LAYOUT
        assert call(B, kv, trees=0, q=B.c_heads(256, 512, 512, -128)) == B.E_LAYOUT
        assert call(B, kv, trees=0, q=B.c_heads(256, 1 << 38, 512, 128)) == B.E_LAYOUT
        assert call(B, kv, trees=0, q=B.c_heads(None, 512, 512, 128)) == B.E_PARAM
        assert call(B, kv, trees=0, hq=0) == B.E_PARAM
    assert _append(B, kv, trees=0, nodes=N(256, None, None, 10, 0, 1)) == B.E_PARAM        # parents without depths
    assert _attend(B, kv, trees=0, nodes=N(256, None, None, 10, 0, 1)) == B.OK             # attention needs none
    for rot in (-16, 8, 24, 144):
        assert _append(B, kv, trees=0, rot=rot) == B.E_PARAM
    assert _append(B, kv, trees=0, rope=None) == B.E_PARAM and _append(B, kv, trees=0, rot=0) == B.E_PARAM
    assert _append(B, kv, trees=0, rows=0) == B.E_PARAM and _append(B, kv, trees=0, rope=260) == B.E_LAYOUT
    assert _append(B, kv, trees=0, qw=258) == B.E_LAYOUT
    for eps in (-1e-6, float("nan"), float("inf")):
        assert _append(B, kv, trees=0, eps=eps) == B.E_PARAM
    assert _attend(B, _kv(B, n_kv_heads=3), trees=0) == B.E_PARAM                          # 4 query heads over 3
    assert _attend(B, _kv(B, n_kv_heads=8), trees=0) == B.E_PARAM
    assert _attend(B, kv, trees=0, hq=128) == B.OK and _attend(B, kv, trees=0, hq=129) == B.E_PARAM  # heads of a key head
    assert B._lib.spec_tree_attend_workspace_bytes(1, 1, 129, 1, 64) == 0
    assert B._lib.spec_tree_attend_workspace_bytes(1, 1, 8, 3, 64) == 0
    assert B._lib.spec_tree_attend_workspace_bytes(1, 1, 8, 1, 96) == 0
    assert _attend(B, kv, trees=0, out=B.c_heads(256, 512, 512, 128)) == B.E_PARAM         # out over q
    assert _attend(B, kv, trees=0, scale=float("nan")) == B.E_PARAM
    assert _attend(B, kv, trees=0, ws=None) == B.E_PARAM and _attend(B, kv, trees=0, ws=264) == B.E_LAYOUT
    for stride in (0, 257):
        assert _commit(B, kv, trees=0, stride=stride) == B.E_PARAM
    assert _commit(B, kv, trees=0, acc=None) == B.E_PARAM and _commit(B, kv, trees=0, node=None) == B.E_PARAM
    assert _commit(B, kv, trees=0, new=None) == B.E_PARAM
    assert _commit(B, kv, trees=0, new=256) == B.E_PARAM                                   # the committed lengths


def test_binding_refuses_tensors_of_another_kind(B):
    k = torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = B.KVCache(k, k.clone(), table, lens)
    assert cache.B == 2 and cache.c().page_size == 16
    for bad in (k.float(), k[0], k.transpose(3, 4)):
        with pytest.raises(B.SpecTreeError):
            B.KVCache(bad, bad, table, lens)
    with pytest.raises(B.SpecTreeError):
        B.KVCache(k, k.transpose(2, 3).contiguous().transpose(2, 3), table, lens)  # k and v in different orders
    with pytest.raises(B.SpecTreeError):
        B.KVCache(k, k, table.long(), lens)
    with pytest.raises(B.SpecTreeError):
        cache.set_lengths(torch.zeros(3, dtype=torch.int32))
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32)
    for bad in (q.half(), q[:1], q[..., :32], q[0]):
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_attend(cache, 0, bad, q.clone(), None, status)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_attend(cache, 0, q, q[:, :, :2], None, status)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_kv_append(cache, 0, q, q, q[:, :, :2], q, None, status)  # keys of four heads, cache of two
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_kv_commit(cache, lens.long(), torch.zeros((2, 4), dtype=torch.int32), lens.clone(), status)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_attend(cache, 0, q, q.clone(), None, status,
                           tree=B.NodeArrays(None, torch.zeros((2, 4), dtype=torch.int32), None))
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_attend(cache, 0, q, q.clone(), None, status, tree=B.NodeArrays(torch.zeros((3, 4), dtype=torch.int32)))


def test_page_tables_whose_rows_overlap_are_refused(B):
    """An expanded table holds one row: read as B rows, it would be read past its end."""
    k, data = torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16), torch.arange(40, dtype=torch.int32)
    lens = torch.zeros(4, dtype=torch.int32)
    for bad in (data[:3].expand(4, -1), data[:3][None].expand(4, -1), data.as_strided((4, 3), (2, 1))):
        with pytest.raises(B.SpecTreeError, match="overlap"):
            B.KVCache(k, k.clone(), bad, lens)
    for good, stride in ((data[:12].view(4, 3), 3), (data.view(4, 10)[:, 2:5], 10), (data[:4].view(4, 1), 1)):
        c = B.KVCache(k, k.clone(), good, lens).c()
        assert (c.max_pages, c.table_stride, c.page_table) == (good.shape[1], stride, good.data_ptr())
    for one in (data[:3].expand(1, -1), data.as_strided((1, 3), (1, 1)), data.as_strided((1, 3), (1 << 40, 1))):
        assert B.KVCache(k, k.clone(), one, lens[:1]).c().table_stride == 3  # the stride of a single row means nothing


class _OnCard(torch.Tensor):
    """A CPU tensor that says it lies on GPU 0."""

    def get_device(self):
        return 0


class _Recorder:
    """Takes the library's place: counts the calls that get through."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def card(B, monkeypatch):
    """(binding, recorder, calls): the entry points' arguments by name, all on GPU 0, and a function for each."""
    rec = _Recorder()
    monkeypatch.setattr(B, "_lib", rec)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 0)
    on = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype).as_subclass(_OnCard)  # noqa: E731
    bf = torch.bfloat16
    pool = dict(kp=on(1, 4, 16, 2, 64, dtype=bf), vp=on(1, 4, 16, 2, 64, dtype=bf), table=on(2, 3), lens=on(2))
    ws = B.AttendWorkspace.__new__(B.AttendWorkspace)
    ws.at, ws.bytes, ws.device = 4096, 1 << 30, 0
    tree = dict(parent=on(2, 9), depth=on(2, 9), n=on(2))

    def cache(a):
        return B.KVCache(a["kp"], a["vp"], a["table"], a["lens"])

    def nodes(a):
        return B.NodeArrays(a["parent"], a["depth"], a["n"])

    append = dict(pool, **tree, q=on(2, 3, 4, 64, dtype=bf), k=on(2, 3, 2, 64, dtype=bf), v=on(2, 3, 2, 64, dtype=bf),
                  out=on(2, 3, 4, 64, dtype=bf), rope=on(9, 64, dtype=torch.float32), qw=on(64, dtype=bf),
                  kw=on(64, dtype=bf), status=on(1))
    attend = dict(pool, **tree, q=append["q"], out=append["out"], ws=ws, status=on(1))
    commit = dict(pool, acc=on(2), node=on(2, 9), new=on(2), status=on(1))
    return rec, [
        (append, lambda a: B.spec_tree_kv_append(cache(a), 0, a["q"], a["k"], a["v"], a["out"], a["rope"], a["status"],
                                                 tree=nodes(a), q_weight=a["qw"], k_weight=a["kw"])),
        (attend, lambda a: B.spec_tree_attend(cache(a), 0, a["q"], a["out"], a["ws"], a["status"], tree=nodes(a))),
        (commit, lambda a: B.spec_tree_kv_commit(cache(a), a["acc"], a["node"], a["new"], a["status"]))]


def test_tensors_on_another_device_are_refused(B, card):
    """Each tensor in turn on the CPU, or the workspace on another GPU: refused before the library is called."""
    rec, calls = card
    for args, call in calls:
        before = rec.calls
        call(args)
        assert rec.calls == before + 1
        for name, x in args.items():
            if name == "ws":
                there = B.AttendWorkspace.__new__(B.AttendWorkspace)
                there.at, there.bytes, there.device = x.at, x.bytes, 1
            else:
                there = x.as_subclass(torch.Tensor)
            with pytest.raises(B.SpecTreeError):
                call(dict(args, **{name: there}))
            assert rec.calls == before + 1, name


def test_caches_off_the_current_gpu_are_refused(B, card, monkeypatch):
    rec, calls = card
    for args, call in calls:
        plain = {k: x if k == "ws" else x.as_subclass(torch.Tensor) for k, x in args.items()}
        with pytest.raises(B.SpecTreeError, match="current GPU"):
            call(plain)                                   # all on the CPU
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    for args, call in calls:
        with pytest.raises(B.SpecTreeError, match="current GPU"):
            call(args)
    assert rec.calls == 0


def test_status_words_of_another_kind_are_refused(B, card):
    """The kernels add bits to a 32-bit word."""
    rec, calls = card
    for args, call in calls:
        for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1, dtype=torch.int64), torch.zeros(1),
                    torch.zeros(0, dtype=torch.int32)):
            with pytest.raises(B.SpecTreeError, match="status"):
                call(dict(args, status=bad.as_subclass(_OnCard)))
        assert rec.calls == 0
    for args, call in calls:
        call(dict(args, status=torch.zeros(3, dtype=torch.uint32).as_subclass(_OnCard)))
    assert rec.calls == 3


def test_structs_match_the_c_header(B, tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = {"spec_tree_kv_t": B.c_kv, "spec_tree_heads_t": B.c_heads, "spec_tree_nodes_t": B.c_nodes}
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "spec_tree.h"', "int main(void) {"]
    for st, cls in fields.items():
        src.append(f'  printf("{st} %zu\\n", sizeof({st}));')
        src += [f'  printf("{st}.{f} %zu\\n", offsetof({st}, {f}));' for f, _ in cls._fields_]
    src += ['  printf("F16 %d\\nS_PAGES %d\\nS_NODES %d\\n", SPEC_TREE_F16, (int)SPEC_TREE_S_PAGES, (int)SPEC_TREE_S_NODES);',
            "  return 0;", "}"]
    c_file, exe = tmp_path / "abi.c", tmp_path / "abi"
    c_file.write_text("\n".join(src) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(c_file), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                       check=True).stdout.splitlines())
    for st, cls in fields.items():
        assert int(got[st]) == ctypes.sizeof(cls), st
        for f, _ in cls._fields_:
            assert int(got[f"{st}.{f}"]) == getattr(cls, f).offset, (st, f)
    assert B._Packed.NODES.size <= ctypes.sizeof(B.c_nodes) and B._Packed.HEADS4.size == 4 * ctypes.sizeof(B.c_heads)
    assert (int(got["F16"]), int(got["S_PAGES"]), int(got["S_NODES"])) == (B.F16, B.S_PAGES, B.S_NODES)


def test_oracle_attention_by_hand():
    """Two tokens and a root with two children, worked out: a child does not see its sibling."""
    k = np.zeros((1, 8, 1, 2))
    v = np.zeros((1, 8, 1, 2))
    k[0, :5, 0] = [[0, 0], [np.log(2), 0], [0, 0], [np.log(3), 0], [np.nan, 0]]
    v[0, :5, 0] = [[1, 0], [0, 1], [4, 0], [0, 2], [np.nan, 9]]
    q = np.zeros((1, 2, 1, 2))
    q[0, :, 0, 0] = 1
    out = O.attend(q, k, v, [[0]], [2], [[-1, 0, 0]], [3], 0, 1.0)[0]
    assert np.allclose(out[0, 0, 0], [5 / 4, 2 / 4])      # weights 1, 2, 1
    assert np.allclose(out[0, 1, 0], [5 / 7, 8 / 7])      # weights 1, 2, 1, 3; node 2 is not seen
    assert O.sees([-1, 0, 0, 1, 3], 4) == [0, 1, 3, 4] and O.sees(None, 2) == [0, 1, 2]


def test_oracle_rotation_keeps_scores_of_equal_distances():
    """Turned queries and keys give scores that depend on the distance alone, in both pairings."""
    rng = np.random.RandomState(0)
    q, k = rng.standard_normal((2, 64))
    a = np.arange(40)[:, None] * 10000.0 ** (-np.arange(16) / 16)
    rope = np.concatenate([np.cos(a), np.sin(a)], 1)
    for inter in (False, True):
        t = lambda x, p: O.turn(x, None, 0.0, rope[p], 32, inter)  # noqa: E731
        assert np.isclose(t(q, 30) @ t(k, 21), t(q, 9) @ t(k, 0))
        assert np.allclose(t(q, 7)[32:], q[32:]) and np.isclose(np.linalg.norm(t(q, 7)), np.linalg.norm(q))


def test_oracle_commit_of_overlapping_slots():
    """A path whose sources are other steps' destinations moves the values that were there before."""
    k = np.arange(8.0).reshape(1, 1, 8, 1, 1)
    got, _, new = O.commit(k, k, [[0]], [1], [3], [[2, 3, 5, -1]])
    assert got[0, 0, :, 0, 0].tolist() == [0, 1, 3, 4, 6, 5, 6, 7] and new.tolist() == [5]


def test_random_trees_are_canonical():
    for seed in range(20):
        parent, depth = kv_cases.random_tree(np.random.RandomState(seed), 61)
        assert parent[0] == -1 and (parent[1:] < np.arange(1, 61)).all() and (np.diff(depth) >= 0).all()
        assert (depth[1:] == depth[parent[1:]] + 1).all() and depth.max() <= 8
