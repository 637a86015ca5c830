"""The 8-bit cache's entry points without a GPU: layout, exports and every
refusal of a bad argument (nothing is launched)."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = ctypes.c_void_p(4096)  # never dereferenced: every case fails validation
ODD = ctypes.c_void_p(4104)


@pytest.fixture(scope="module")
def lrkv():
    from rank_kv_cache_lrkv_b200 import lrkv as m
    return m


def _desc(lrkv, **kw):
    base = dict(batch=2, num_kv_heads=2, head_dim=128, code=0, num_pages=4, max_pages_per_seq=2,
                pages=16, block_table=16, tail=16, seq_len=16, append_counter=16, error=16)
    base.update(kw)
    return lrkv.QuantDesc(**base)


def test_struct_and_constants_match_the_header(lrkv, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(
        '#include <stdio.h>\n#include <stddef.h>\n#include "lrkv.h"\n'
        'int main(void){printf("%zu %zu %zu %zu %d %d %d %d", sizeof(lrkv_quant_cache),'
        ' offsetof(lrkv_quant_cache, pages), offsetof(lrkv_quant_cache, tail),'
        ' offsetof(lrkv_quant_cache, error), LRKV_CODE_INT8, LRKV_CODE_E4M3, LRKV_QUANT_TAIL,'
        ' LRKV_QUANT_SLAB_BYTES);return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    D = lrkv.QuantDesc
    assert list(map(int, subprocess.check_output([str(exe)]).split())) == [
        ctypes.sizeof(D), D.pages.offset, D.tail.offset, D.error.offset,
        lrkv.QUANT_CODES["int8"], lrkv.QUANT_CODES["e4m3"], lrkv.QUANT_TAIL,
        lrkv.QUANT_SLAB_BYTES]


@pytest.mark.parametrize("field,value,status", [
    ("head_dim", 64, -2), ("code", 2, -2), ("code", -1, -2), ("batch", 0, -1), ("batch", 1025, -1),
    ("num_kv_heads", 0, -1), ("num_kv_heads", 32768, -1), ("num_pages", 0, -1),
    ("max_pages_per_seq", 0, -1), ("max_pages_per_seq", (1 << 25), -1), ("pages", 0, -1),
    ("pages", 8, -1), ("tail", 0, -1), ("tail", 24, -1), ("block_table", 0, -1),
    ("seq_len", 0, -1), ("append_counter", 0, -1), ("error", 0, -1)])
def test_every_call_refuses_a_bad_cache(lrkv, field, value, status):
    d, L = ctypes.byref(_desc(lrkv, **{field: value})), lrkv._lib
    assert L.lrkv_quant_append(d, FAKE, FAKE, 4, None, 512, 512, 128, None) == status
    assert L.lrkv_quant_read(d, None, 4, FAKE, FAKE, 0, 512, 512, 128, None) == status
    assert L.lrkv_quant_attn_workspace_bytes(d, 4, 1) == 0
    assert L.lrkv_quant_attn(d, FAKE, 4, 1, None, 512, 128, 128, 0.1, FAKE, 512, 128, 128, FAKE,
                             1 << 30, None) == status


def test_append_refuses_bad_calls(lrkv):
    d, L = ctypes.byref(_desc(lrkv)), lrkv._lib

    def call(k=FAKE, v=FAKE, n=4, ss=512, hs=512, ts=128, desc=d):
        return L.lrkv_quant_append(desc, k, v, n, None, ss, hs, ts, None)

    assert call(desc=None) == -1
    assert call(n=-1) == -1
    assert call(n=0) == 0
    assert call(k=None) == -1 and call(v=None) == -1
    assert call(k=ODD) == -1 and call(v=ODD) == -1
    assert call(ss=4) == -1 and call(hs=12) == -1 and call(ts=129) == -1
    assert call(n=129) == -3  # 2 pages x 64 tokens


def test_read_refuses_bad_calls(lrkv):
    d, L = ctypes.byref(_desc(lrkv)), lrkv._lib

    def call(k=FAKE, v=FAKE, n=4, dtype=0, ss=512, hs=512, ts=128):
        return L.lrkv_quant_read(d, None, n, k, v, dtype, ss, hs, ts, None)

    assert L.lrkv_quant_read(None, None, 4, FAKE, FAKE, 0, 0, 0, 0, None) == -1
    assert call(n=-1) == -1 and call(n=0) == 0
    assert call(dtype=2) == -2 and call(dtype=-1) == -2
    assert call(k=None) == -1 and call(v=ODD) == -1
    assert call(ts=132) == -1 and call(ts=130, dtype=1) == -1


def test_attention_refuses_bad_calls(lrkv):
    d, L = ctypes.byref(_desc(lrkv)), lrkv._lib

    def call(q=FAKE, o=FAKE, ws=FAKE, hq=4, n=1, nb=1 << 30, q3=(512, 128, 128),
             o3=(512, 128, 128), desc=d):
        return L.lrkv_quant_attn(desc, q, hq, n, None, *q3, 0.1, o, *o3, ws, nb, None)

    assert call(desc=None) == -1
    assert call(hq=3) == -1 and call(hq=0) == -1 and call(n=-1) == -1
    assert call(hq=258) == -2                       # 129 query heads per KV head
    assert call(n=1 << 30) == -2                    # rows past 32 bits
    many = ctypes.byref(_desc(lrkv, batch=1024, max_pages_per_seq=1 << 20))
    assert call(desc=many) == -2                    # blocks past 32 bits
    long = ctypes.byref(_desc(lrkv, batch=1, num_kv_heads=1, max_pages_per_seq=65536))
    assert call(hq=8, n=1 << 22, desc=long) == -2   # a unit's row tiles x blocks past 32 bits
    assert L.lrkv_quant_attn_workspace_bytes(long, 8, 1 << 22) == 0
    assert call(n=0) == 0
    assert call(q=None) == -1 and call(o=None) == -1 and call(ws=None) == -1
    assert call(q=ODD) == -1 and call(o=ODD) == -1 and call(ws=ODD) == -1
    for i in range(3):
        bad = [512, 128, 128]
        bad[i] += 4
        assert call(q3=bad) == -1 and call(o3=bad) == -1
    assert L.lrkv_quant_attn_workspace_bytes(d, 3, 1) == 0
    assert L.lrkv_quant_attn_workspace_bytes(d, 4, -1) == 0


def test_the_binding_refuses_bad_tensors(lrkv):
    c = lrkv.QuantCache(2, 2, 100, device="cpu")
    assert c.max_pages == 2 and c.pages.shape == (4, 2, 16416)
    with pytest.raises(ValueError):
        lrkv.QuantCache(1, 1, 10, code="int4", device="cpu")
    k = torch.zeros(2, 2, 3, 128, dtype=torch.bfloat16)
    bad = [k.float(), k[:1], k[:, :1], k[..., :64], k.transpose(2, 3), k[:, :, 0],
           k.to("meta"), torch.zeros(2, 2, 3, 256, dtype=torch.bfloat16)[..., ::2]]
    for x in bad:
        with pytest.raises(ValueError):
            lrkv.quant_append(c, x, k)
        with pytest.raises(ValueError):
            lrkv.quant_append(c, k, x)
    for n_new in (torch.zeros(2), torch.zeros(3, dtype=torch.int32),
                  torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            lrkv.quant_append(c, k, k, n_new=n_new)
        with pytest.raises(ValueError):
            lrkv.quant_read(c, k, k, first=n_new)
        with pytest.raises(ValueError):
            lrkv.quant_attn(c, k, 0.1, k, torch.zeros(64, dtype=torch.uint8), n_q=n_new)
    with pytest.raises(ValueError):   # one shape, two layouts
        lrkv.quant_append(c, k, torch.zeros(2, 3, 2, 128, dtype=torch.bfloat16).transpose(1, 2))
    for x in (k.half(), k.expand(2, 2, 3, 128)[:, :, :1].expand(2, 2, 3, 128)):
        with pytest.raises(ValueError):
            lrkv.quant_read(c, x, x)
    q = torch.zeros(2, 4, 1, 128, dtype=torch.bfloat16)
    ws = torch.zeros(64, dtype=torch.uint8)
    for args in ((q, 0.1, q[:, :, 0], ws), (q.float(), 0.1, q.float(), ws),
                 (q, 0.1, q[:1].expand(2, 4, 1, 128), ws), (q, 0.1, q, ws.float()),
                 (q[0], 0.1, q[0], ws), (q, 0.1, q, ws)):
        with pytest.raises(ValueError):
            lrkv.quant_attn(c, *args)
