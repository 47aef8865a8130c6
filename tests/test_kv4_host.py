"""The key-value cache in 4 bits and the page pool without a GPU: refusals before any launch, structures, the oracle."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as O4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
VP = ctypes.c_void_p


@pytest.fixture(scope="module")
def B():
    from dynamic_tree_speculative_gb300 import binding
    return binding


def _kv4(B, scale=256, scale_strides=(0, 512, 512), **kw):
    c = B.c_kv(256, 256, 256, 256, 0, 2048, 128, 128, B.BF16, 1, 4, 16, 1, 128, 8, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return B.c_kv4(c, scale, *scale_strides)


def _calls(B, kv, trees=0, layer=0, hq=4, q=None):
    """Return codes of append, attend, commit and read (the layer is not commit's)."""
    r, h, n = ctypes.byref, B.c_heads(256, 512, 512, 128), B.c_nodes(None, None, None, 0, 0, 1)
    other = B.c_heads(4096, 512, 512, 128)
    q = q or h
    return (B._lib.spec_tree_kv4_append(trees, r(kv), layer, r(n), hq, r(q), r(h), r(h), r(h), VP(256), 100, 64, 0, None,
                                        None, 1e-6, None, None),
            B._lib.spec_tree_kv4_attend(trees, r(kv), layer, r(n), hq, r(q), r(other), 0.1, VP(256), 1 << 40, None, None),
            B._lib.spec_tree_kv4_commit(trees, r(kv), VP(256), VP(256), 9, VP(512), None, None),
            B._lib.spec_tree_kv4_read(trees, r(kv), layer, None, None, 5, r(q), r(other), None, None))


# trees = 0: the checks alone run, no launch follows
def test_accepted_arguments(B):
    assert _calls(B, _kv4(B)) == (B.OK,) * 4
    assert _calls(B, _kv4(B, dtype=B.F16, head_dim=64)) == (B.OK,) * 4


@pytest.mark.parametrize("field,value,rc", [
    ("dtype", 1, "E_LAYOUT"), ("head_dim", 96, "E_PARAM"), ("page_size", 4, "E_PARAM"), ("page_size", 24, "E_PARAM"),
    ("n_pages", 0, "E_PARAM"), ("max_pages", 9, "E_PARAM"), ("k", 264, "E_LAYOUT"), ("v", None, "E_PARAM"),
    ("page_table", None, "E_PARAM"), ("token_stride", 136, "E_LAYOUT"), ("token_stride", 144, "E_LAYOUT"),
    ("head_stride", -128, "E_LAYOUT"), ("page_stride", 2064, "E_LAYOUT"),
])
def test_bad_caches(B, field, value, rc):
    """Strides of a cache in 4 bits are multiples of 32 codes: 16 bytes."""
    assert _calls(B, _kv4(B, **{field: value})) == (getattr(B, rc),) * 4


def test_bad_scales(B):
    assert _calls(B, _kv4(B, scale=None)) == (B.E_PARAM,) * 4
    assert _calls(B, _kv4(B, scale=264)) == (B.E_LAYOUT,) * 4
    for bad in ((4, 512, 512), (0, 516, 512), (0, 512, 60), (0, -512, 512), (0, 1 << 38, 64)):
        assert _calls(B, _kv4(B, scale_strides=bad)) == (B.E_LAYOUT,) * 4


def test_bad_calls(B):
    kv = _kv4(B)
    r, h, other = ctypes.byref, B.c_heads(256, 512, 512, 128), B.c_heads(4096, 512, 512, 128)
    assert _calls(B, kv, trees=-1) == (B.E_PARAM,) * 4 and _calls(B, kv, trees=65536) == (B.E_PARAM,) * 4
    a = _calls(B, kv, layer=1)
    assert (a[0], a[1], a[3]) == (B.E_PARAM,) * 3
    assert _calls(B, kv, q=B.c_heads(264, 512, 512, 128))[3] == B.E_LAYOUT
    read = B._lib.spec_tree_kv4_read
    for count in (0, -1, (1 << 20) + 1):
        assert read(0, r(kv), 0, None, None, count, r(h), r(other), None, None) == B.E_PARAM
    assert read(0, r(kv), 0, None, None, 5, r(h), r(h), None, None) == B.E_PARAM       # keys over values
    assert read(2000, r(kv), 0, None, None, 1 << 20, r(h), r(other), None, None) == B.E_PARAM  # vectors past 2^30
    assert read(0, r(_kv4(B, seq_len=None)), 0, None, None, 5, r(h), r(other), None, None) == B.OK
    assert B._lib.spec_tree_kv4_attend(0, r(_kv4(B, seq_len=None)), 0, r(B.c_nodes(None, None, None, 0, 0, 1)), 4, r(h),
                                       r(other), 0.1, VP(256), 1 << 40, None, None) == B.E_PARAM
    assert read(0, None, 0, None, None, 5, r(h), r(other), None, None) == B.E_PARAM


def test_bad_pools(B):
    good = dict(page_table=256, held=256, free_pages=256, n_free=256, scratch=256, n_pages=9, page_size=16, max_pages=4,
                table_stride=4)

    def both(trees=0, lens=256, keep=256, count=3, slots=None, **kw):
        p = B.c_pages(**dict(good, **kw))
        return (B._lib.spec_tree_kv_reserve(trees, ctypes.byref(p), VP(lens), None, count, VP(slots), None, None),
                B._lib.spec_tree_kv_release(trees, ctypes.byref(p), VP(keep), None, None))

    assert both() == (B.OK, B.OK) and both(table_stride=9) == (B.OK, B.OK)
    for bad in (dict(page_table=None), dict(held=None), dict(free_pages=None), dict(n_free=None), dict(scratch=None),
                dict(n_pages=0), dict(page_size=4), dict(page_size=48), dict(page_size=1 << 17), dict(max_pages=0),
                dict(max_pages=5), dict(max_pages=1 << 27, table_stride=1 << 27), dict(trees=-1), dict(trees=65536)):
        assert both(**bad) == (B.E_PARAM, B.E_PARAM), bad
    assert both(lens=None)[0] == B.E_PARAM and both(keep=None)[1] == B.E_PARAM
    assert both(count=0)[0] == B.E_PARAM and both(count=(1 << 20) + 1)[0] == B.E_PARAM
    assert both(slots=260)[0] == B.E_LAYOUT


def test_structs_match_the_c_header(B, tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = {"spec_tree_kv4_t": B.c_kv4, "spec_tree_pages_t": B.c_pages}
    src = ["#include <stddef.h>", "#include <stdio.h>", '#include "spec_tree.h"', "int main(void) {"]
    for st, cls in fields.items():
        src.append(f'  printf("{st} %zu\\n", sizeof({st}));')
        src += [f'  printf("{st}.{f} %zu\\n", offsetof({st}, {f}));' for f, _ in cls._fields_]
    src += ["  return 0;", "}"]
    c_file, exe = tmp_path / "abi.c", tmp_path / "abi"
    c_file.write_text("\n".join(src) + "\n")
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(c_file), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for st, cls in fields.items():
        assert int(got[st]) == ctypes.sizeof(cls), st
        for f, _ in cls._fields_:
            assert int(got[f"{st}.{f}"]) == getattr(cls, f).offset, (st, f)


def test_binding_refuses_tensors_of_another_kind(B):
    k = torch.zeros((1, 4, 16, 2, 32), dtype=torch.uint8)
    scale = torch.zeros((1, 4, 2, 16, 4), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = B.KVCache4(k, k.clone(), scale, table, lens)
    assert (cache.B, cache.c().kv.page_size, cache.c().kv.head_dim, cache.c().kv.token_stride) == (2, 16, 64, 128)
    for bad in (k.to(torch.int8), k[0], k.transpose(3, 4)):
        with pytest.raises(B.SpecTreeError):
            B.KVCache4(bad, bad, scale, table, lens)
    for bad in (scale.float(), scale[:, :3], scale.transpose(2, 3), scale.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(B.SpecTreeError):
            B.KVCache4(k, k.clone(), bad, table, lens)
    with pytest.raises(B.SpecTreeError):
        B.KVCache4(k, k, scale, table.long(), lens)
    with pytest.raises(B.SpecTreeError):
        B.KVCache4(k, k, scale, table[0].expand(2, -1), lens)
    with pytest.raises(B.SpecTreeError):
        cache.set_lengths(lens[:1])
    q, status = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    kv = torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16)
    half = B.KVCache(torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16), torch.zeros((1, 4, 16, 2, 64), dtype=torch.bfloat16),
                     table, lens)
    for mine, theirs in ((cache, (B.spec_tree_kv_append, B.spec_tree_attend, B.spec_tree_kv_commit)),
                         (half, (B.spec_tree_kv4_append, B.spec_tree_kv4_attend, B.spec_tree_kv4_commit))):
        with pytest.raises(B.SpecTreeError, match="cache must be"):
            theirs[0](mine, 0, q, kv, kv, q, None, status)
        with pytest.raises(B.SpecTreeError, match="cache must be"):
            theirs[1](mine, 0, q, q.clone(), None, status)
        with pytest.raises(B.SpecTreeError, match="cache must be"):
            theirs[2](mine, lens, torch.zeros((2, 4), dtype=torch.int32), lens.clone(), status)
    with pytest.raises(B.SpecTreeError, match="cache must be"):
        B.spec_tree_kv4_read(half, 0, kv, kv.clone(), status)
    for bad in (q.half(), q[:1], q[..., :32], q[0]):
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_kv4_attend(cache, 0, bad, q.clone(), None, status)
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_kv4_read(cache, 0, bad, kv, status)
    with pytest.raises(B.SpecTreeError, match="current GPU"):
        B.spec_tree_kv4_read(cache, 0, kv, kv.clone(), status)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_kv4_read(cache, 0, kv, kv.clone(), status, first=lens.long())


def test_binding_refuses_pools_of_another_kind(B):
    i32 = dict(dtype=torch.int32)
    table, held, free, one = torch.zeros((2, 3), **i32), torch.zeros(2, **i32), torch.zeros(9, **i32), torch.zeros(1, **i32)
    pool = B.PagePool(9, 16, 2, 3, table, held, free, one)
    assert (pool.c().n_pages, pool.c().table_stride, pool.c().held) == (9, 3, held.data_ptr())
    assert B.PagePool(9, 16, 2, 3, device="cpu").free.tolist() == list(range(8, -1, -1))
    for bad in ((table, held, free, None), (table[:, :2], held, free, one), (table, held[:1], free, one),
                (table, held, free[:8], one), (table, held, free, held), (table.long(), held, free, one),
                (table[:1].expand(2, -1), held, free, one)):
        with pytest.raises(B.SpecTreeError):
            B.PagePool(9, 16, 2, 3, *bad)
    status = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_kv_reserve(pool, held[:1], 4, status)
    for bad in (torch.zeros((2, 4), dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int64), torch.zeros((4, 2), dtype=torch.int64).T):
        with pytest.raises(B.SpecTreeError):
            B.spec_tree_kv_reserve(pool, held, 4, status, slots=bad)
    with pytest.raises(B.SpecTreeError):
        B.spec_tree_kv_release(pool, held.long(), status)
    with pytest.raises(B.SpecTreeError, match="current GPU"):
        B.spec_tree_kv_release(pool, held, status)


class _OnCard(torch.Tensor):
    """A CPU tensor that says it lies on GPU 0."""

    def get_device(self):
        return 0


def test_tensors_on_another_device_are_refused(B, monkeypatch):
    """Each tensor in turn on the CPU, the rest on the GPU: refused before the library is called."""
    class Recorder:
        calls = 0

        def __getattr__(self, name):
            def call(*args):
                Recorder.calls += 1
                return 0
            return call

    monkeypatch.setattr(B, "_lib", Recorder())
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_raw_stream", lambda device: 0)
    on = lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype).as_subclass(_OnCard)  # noqa: E731
    bf, u8 = torch.bfloat16, torch.uint8
    base = dict(k4=on(1, 4, 16, 2, 32, dtype=u8), v4=on(1, 4, 16, 2, 32, dtype=u8), sc=on(1, 4, 2, 16, 4, dtype=bf), table=on(2, 3),
                lens=on(2), status=on(1))
    cache = lambda a: B.KVCache4(a["k4"], a["v4"], a["sc"], a["table"], a["lens"])  # noqa: E731
    q, k = on(2, 3, 4, 64, dtype=bf), on(2, 3, 2, 64, dtype=bf)
    pages = dict(table=on(2, 3), held=on(2), free=on(9), n_free=on(1), lens=on(2), status=on(1))

    def pool(a):
        p = B.PagePool(9, 16, 2, 3, a["table"], a["held"], a["free"], a["n_free"])
        return p

    calls = [
        (dict(base, q=q, k=k, v=k.clone(), out=q.clone()),
         lambda a: B.spec_tree_kv4_append(cache(a), 0, a["q"], a["k"], a["v"], a["out"], None, a["status"])),
        (dict(base, acc=on(2), node=on(2, 9), new=on(2)),
         lambda a: B.spec_tree_kv4_commit(cache(a), a["acc"], a["node"], a["new"], a["status"])),
        (dict(base, k=k, v=k.clone(), first=on(2), counts=on(2)),
         lambda a: B.spec_tree_kv4_read(cache(a), 0, a["k"], a["v"], a["status"], a["first"], a["counts"])),
        (dict(pages, n=on(2), slots=on(2, 4, dtype=torch.int64)),
         lambda a: B.spec_tree_kv_reserve(pool(a), a["lens"], 4, a["status"], a["n"], a["slots"])),
        (pages, lambda a: B.spec_tree_kv_release(pool(a), a["lens"], a["status"]))]
    for args, call in calls:
        before = Recorder.calls
        call(args)
        assert Recorder.calls == before + 1
        for name, x in args.items():
            with pytest.raises(B.SpecTreeError):
                call(dict(args, **{name: x.as_subclass(torch.Tensor)}))
            assert Recorder.calls == before + 1, name


# ------------------------------------------------------------------ the oracle ---

def test_quantised_vectors_by_hand():
    x = np.array([-1.0, 14.0, 0.25, 3.5, 4.5, -1.0, 13.75, 6.0])
    codes, s, z = O4.quantise(x)                     # scale 1: 0.25 is 1.25 steps up, 3.5 and 4.5 are ties
    assert (float(s), float(z)) == (1.0, -1.0) and codes.tolist() == [0, 15, 1, 4, 6, 0, 15, 7]
    codes, s, z = O4.quantise(np.full(8, 2.5))
    assert (float(s), float(z)) == (0.0, 2.5) and not codes.any()
    for bad in (np.nan, np.inf):
        codes, s, z = O4.quantise(np.where(np.arange(8) == 3, bad, x))
        assert np.isnan(s) and np.isnan(z) and not codes.any()
    assert np.isnan(O4.quantise(np.array([3e38, -3e38]))[1])
    assert O4.towards_zero(np.array([1.9999, 257.0]), 8, -133).tolist() == [1.9921875, 256.0]
    data = O4.pack(np.arange(16, dtype=np.uint8))
    assert data.tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] and O4.unpack(data).tolist() == list(range(16))


@pytest.mark.parametrize("dtype,bits", [(torch.bfloat16, 8), (torch.float16, 11)])
def test_quantised_vectors_are_near(dtype, bits):
    """Within half a step, but for what the scale, rounded towards zero, falls short by: 15 steps of 2^(1 - bits) each; and
    never past the largest element."""
    x = torch.randn((500, 128), generator=torch.Generator().manual_seed(0)).to(dtype).double().numpy()
    codes, s, z = O4.quantise(x, bits)
    y = O4.values(codes, s, z)
    assert (np.abs(y - x) <= s[:, None] * (0.5 + 15 * 2.0 ** (1 - bits)) * (1 + 1e-6)).all()
    assert (y <= x.max(-1, keepdims=True) * (1 + 2.0 ** -22)).all() and (y >= x.min(-1, keepdims=True)).all()
    assert torch.equal(torch.from_numpy(s).to(dtype).double(), torch.from_numpy(s))


def test_page_pool_by_hand():
    p = O4.Pages(3, 6, 16, 4, [5, 4, 3, 2, 1, 0])
    slots, short = p.reserve([0, 15, -1], 2)
    assert not short and p.rows == [[0], [1, 2], []] and slots == [[0, 1], [31, 32], [-1, -1]]
    slots, short = p.reserve([40, 60, 0], 5)         # 45 slots: two more; 65: past four pages; one
    assert short and p.rows == [[0, 3, 4], [1, 2], [5]] and slots[1] == [-1] * 5 and slots[2] == [80, 81, 82, 83, 84]
    before = list(p.stack), [list(r) for r in p.rows]
    p.release([45, 32, 0])
    assert p.stack == [5] and p.rows == [[0, 3, 4], [1, 2], []]
    assert not p.reserve([0, 0, 0], 1)[1] and (p.stack, p.rows) == before
