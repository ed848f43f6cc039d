"""Host-side checks of the paged-cache entry points (no GPU): structure
layout, workspace sizes, and the refusals that come back before anything
touches a device, from the C ABI and from the Python binding."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import top_moe_block_b200 as ZB
from synthetic import get_config
from top_moe_block_b200 import _abi, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, MISALIGNED, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
P = C.c_void_p(1 << 16)          # stands for a device pointer: every call below is refused before it is used
FREE = C.c_void_p(1 << 17)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _abi.lib()


def _cfg(**kw):
    return ZB.make_config(get_config("prefill_4k").with_(**kw))


def _kv(n_pages=8, page=64, k=1 << 16, v=1 << 16):
    s = _abi.zaya_paged_kv()
    s.k_pages, s.v_pages, s.n_pages, s.page_size = k, v, n_pages, page
    return s


def test_struct_layout_matches_header(tmp_path):
    structs = [("zaya_paged_kv", _abi.zaya_paged_kv), ("zaya_paged_state", _abi.zaya_paged_state)]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "zaya.h"', 'int main(void){']
    for name, ct in structs:
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in ct._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "a")], check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "a")], capture_output=True, text=True).stdout.splitlines())
    for name, ct in structs:
        assert int(got[name]) == C.sizeof(ct)
        for f, _ in ct._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(ct, f).offset


def _plan(lib, B=4, T=16, ctx=P, new=P, table=P, max_pages=8, free=P, n_pages=64, n_in=P, n_out=P, page=16, cu=P,
          seq=FREE, slot=P, pos=P, row=P, ws=P, ws_bytes=256):
    return lib.zaya_paged_plan(B, T, ctx, new, None, table, max_pages, free, n_pages, n_in, n_out, page, cu, seq, slot,
                               pos, row, ws, ws_bytes, None)


@pytest.mark.parametrize("kw, code", [
    (dict(B=0), INVALID), (dict(T=0), INVALID), (dict(max_pages=0), INVALID), (dict(n_pages=0), INVALID),
    (dict(seq=P), INVALID), (dict(ws=None), INVALID), (dict(B=4097), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(page=24), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(page=0), UNSUPPORTED),
    (dict(n_pages=1 << 27), UNSUPPORTED), (dict(ws=C.c_void_p(65536 + 128)), MISALIGNED), (dict(ws_bytes=255), WORKSPACE)]
    + [({k: None}, INVALID) for k in ("ctx", "new", "table", "free", "n_in", "n_out", "cu", "seq", "slot", "pos", "row")])
def test_plan_refuses(lib, kw, code):
    assert _plan(lib, **kw) == code


def _store(lib, cfg, T=4, k=P, ks=256, v=P, vs=256, slot=P, kv=None, ws=P, ws_bytes=256):
    return lib.zaya_paged_store(C.byref(cfg), T, k, ks, v, vs, slot, C.byref(kv or _kv()), ws, ws_bytes, None)


def test_store_refuses(lib):
    c = _cfg()
    for kw, code in [(dict(T=0), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slot=None), INVALID),
                     (dict(ks=248), INVALID), (dict(vs=0), INVALID), (dict(ks=260), MISALIGNED),
                     (dict(k=C.c_void_p(65538)), MISALIGNED), (dict(kv=_kv(n_pages=0)), INVALID),
                     (dict(kv=_kv(k=None)), INVALID), (dict(kv=_kv(page=48)), UNSUPPORTED),
                     (dict(kv=_kv(v=65544)), MISALIGNED), (dict(kv=_kv(n_pages=1 << 25)), UNSUPPORTED),
                     (dict(ws=None), INVALID), (dict(ws_bytes=0), WORKSPACE)]:
        assert _store(lib, c, **kw) == code, kw
    assert _store(lib, _cfg(head_dim=96)) == UNSUPPORTED
    assert _store(lib, _cfg(n_q=6, n_kv=2)) == UNSUPPORTED
    assert _store(lib, _cfg(n_q=9, n_kv=2)) == INVALID
    assert _store(lib, _cfg(kv_fp8=2)) == INVALID


def test_attention_refuses(lib):
    c = _cfg()
    n = ZB.zaya_attention_workspace_size(c)
    assert n >= 256 + 4096
    assert ZB.zaya_attention_workspace_size(_cfg(head_dim=96)) == 0

    def paged(window=64, B=2, T=4, q=P, qs=1024, cu=P, seq=P, table=P, max_pages=4, kv=None, out=P, os_=1024, ws=P,
              ws_bytes=n, cfg=c):
        return lib.zaya_paged_attention(C.byref(cfg), window, B, T, q, qs, cu, seq, table, max_pages,
                                        C.byref(kv or _kv()), out, os_, ws, ws_bytes, None)

    def packed(window=64, B=2, T=4, q=P, qs=1024, k=P, ks=256, v=P, vs=256, cu=P, out=P, os_=1024, ws=P, ws_bytes=n, cfg=c):
        return lib.zaya_packed_attention(C.byref(cfg), window, B, T, q, qs, k, ks, v, vs, cu, out, os_, ws, ws_bytes, None)

    both = [(dict(window=0), INVALID), (dict(window=-3), INVALID), (dict(B=0), INVALID), (dict(T=0), INVALID),
            (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(cu=None), INVALID), (dict(qs=1016), INVALID),
            (dict(os_=1028), MISALIGNED), (dict(q=C.c_void_p(65544)), MISALIGNED), (dict(ws=None), INVALID),
            (dict(ws=C.c_void_p(65536 + 16)), MISALIGNED), (dict(ws_bytes=n - 1), WORKSPACE), (dict(B=4097), UNSUPPORTED),
            (dict(T=1 << 24), UNSUPPORTED)]
    for kw, code in both:
        assert paged(**kw) == code, kw
        assert packed(**kw) == code, kw
    for kw, code in [(dict(seq=None), INVALID), (dict(table=None), INVALID), (dict(max_pages=0), INVALID),
                     (dict(kv=_kv(page=40)), UNSUPPORTED), (dict(kv=_kv(k=65537)), MISALIGNED)]:
        assert paged(**kw) == code, kw
    for kw, code in [(dict(k=None), INVALID), (dict(ks=128), INVALID), (dict(vs=264 + 4), MISALIGNED)]:
        assert packed(**kw) == code, kw
    assert paged(cfg=_cfg(n_q=32, n_kv=2)) == UNSUPPORTED


def test_block_paged_refuses(lib):
    c = _cfg()
    n = ZB.zaya_paged_workspace_size(c, 4, 32)
    assert n > 0
    assert ZB.zaya_paged_workspace_size(c, 4, 64) > n
    assert ZB.zaya_paged_workspace_size(c, 0, 32) == 0 and ZB.zaya_paged_workspace_size(c, 4, 0) == 0
    w = _abi.zaya_block_weights()
    for name in _abi.WEIGHT_FIELDS:
        setattr(w, name, 1 << 16)

    def call(cfg=c, bidx=1, B=4, T=32, hidden=P, cu=P, seq=P, slot=P, row=P, table=P, max_pages=4, fresh=0, rin=P,
             rout=FREE, kv=None, conv=1 << 16, hs=1 << 16, ws=P, ws_bytes=n):
        s = _abi.zaya_paged_state()
        s.kv, s.conv_state, s.prev_hs = kv or _kv(), conv, hs
        return lib.zaya_block_paged(C.byref(cfg), C.byref(w), bidx, B, T, hidden, cu, seq, slot, row, table, max_pages,
                                    fresh, rin, rout, C.byref(s), None, ws, ws_bytes, None)

    for kw, code in [(dict(B=0), INVALID), (dict(T=0), INVALID), (dict(hidden=None), INVALID), (dict(cu=None), INVALID),
                     (dict(seq=None), INVALID), (dict(slot=None), INVALID), (dict(row=None), INVALID),
                     (dict(table=None), INVALID), (dict(max_pages=0), INVALID), (dict(fresh=2), INVALID),
                     (dict(rin=None), INVALID), (dict(rout=P), INVALID), (dict(rout=None), INVALID),
                     (dict(bidx=-1), INVALID), (dict(conv=None), INVALID), (dict(hs=None), INVALID),
                     (dict(conv=65544), MISALIGNED), (dict(hidden=C.c_void_p(65540)), MISALIGNED),
                     (dict(kv=_kv(page=100)), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(ws_bytes=n - 256), WORKSPACE),
                     (dict(cfg=_cfg(kv_ring=1)), UNSUPPORTED),
                     (dict(cfg=ZB.make_config(get_config("prefill_4k_conv2"))), UNSUPPORTED)]:
        assert call(**kw) == code, kw


def test_binding_checks_tensors():
    """Wrong types, shapes, layouts and devices are a ValueError, before the library is called."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c = _cfg()
    with pytest.raises(ValueError):
        ZB.make_paged_kv(torch.zeros(2, 2, 16, 128), torch.zeros(2, 2, 16, 128))
    with pytest.raises(ValueError):
        ZB.make_paged_kv(torch.zeros(2, 2, 16, 128, dtype=torch.uint8), torch.zeros(3, 2, 16, 128, dtype=torch.uint8))
    pages = torch.zeros(2, 2, 16, 128, dtype=torch.bfloat16)
    kv = ZB.make_paged_kv(pages, pages.clone())
    rows = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):     # host tensors
        ZB.zaya_paged_store(c, rows, rows, i(4), kv, ws)
    with pytest.raises(ValueError):
        ZB.zaya_paged_plan(i(2), i(2), None, i(2, 4), i(8), i(1), i(1), 16, i(3), i(2), i(4), i(4), i(4), ws)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ZB.zaya_paged_attention(c, 8, q, i(3), i(2), i(2, 4), kv, q.clone(), ws)
    with pytest.raises(ValueError):
        ZB.zaya_packed_attention(c, 8, q, rows, rows, i(3), q.clone(), ws)


def test_binding_is_rebuilt_for_another_torch_or_interpreter(tmp_path, monkeypatch):
    assert build._fast_up_to_date()         # as the fixture left it
    fast, stamp = tmp_path / "_fast.so", tmp_path / "_fast.stamp"
    fast.write_bytes(b"")
    monkeypatch.setattr(build, "FAST", str(fast))
    monkeypatch.setattr(build, "FAST_STAMP", str(stamp))
    assert not build._fast_up_to_date()     # a module of unknown origin
    stamp.write_text(build._fast_stamp())
    assert build._fast_up_to_date()
    for change in (lambda m: m.setattr(torch, "__version__", "9.9.9"), lambda m: m.setattr(build, "_fast_flags", lambda: ["-O3"]),
                   lambda m: m.setattr("sysconfig.get_config_var", lambda name: "cpython-999")):
        with monkeypatch.context() as m:
            change(m)
            assert not build._fast_up_to_date()
    os.utime(fast, (0, 0))
    assert not build._fast_up_to_date()     # older than its source


def test_binding_that_does_not_load_says_why(tmp_path, monkeypatch):
    monkeypatch.setattr(_abi, "_fast", None)
    monkeypatch.delattr(ZB, "_fast", raising=False)
    monkeypatch.setitem(sys.modules, "top_moe_block_b200._fast", None)     # stands for an undefined symbol
    with pytest.raises(ImportError, match="does not load: import of top_moe_block_b200._fast halted"):
        _abi.fast()
    monkeypatch.setattr(_abi, "FAST_PATH", str(tmp_path / "_fast.so"))
    with pytest.raises(ImportError, match="not built"):
        _abi.fast()
