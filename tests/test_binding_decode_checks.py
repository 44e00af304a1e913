"""What the binding refuses of the attention calls over 4-bit pools and of cross attention before they reach
the library: a short output, and for the decode calls any tensor of another device, too small or a workspace
that is not on the device.  The library is a stand-in: a call that passes the checks is counted."""
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa
from pagedattention_kv_cache_pa_b200 import binding
from tests.test_binding_checks import DESC, POOL, ROWS, Fake

NEW = 3 * 2 * 64
OPTS = pa.DecodeOptions(kv_dtype=pa.PA_KV_E2M1, k_scale=1.0, v_scale=1.0)


@pytest.fixture(autouse=True)
def library(monkeypatch):
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(binding, "_device", lambda: 0)
    monkeypatch.setattr(binding, "lib", Lib())
    return calls


class Space(Fake):
    def element_size(self):
        return self.dtype.itemsize


def decode(call, opts=OPTS, **other):
    cache = torch.uint8 if opts is not None else torch.bfloat16
    n = POOL * 9 // 16 if opts is not None else POOL
    a = dict(q=Fake(torch.bfloat16, ROWS), out=Fake(torch.bfloat16, ROWS), k=Fake(torch.bfloat16, NEW),
             v=Fake(torch.bfloat16, NEW), k_cache=Fake(cache, n), v_cache=Fake(cache, n), tables=Fake(torch.int32, 6),
             lens=Fake(torch.int32, 3), workspace=Space(torch.uint8, 1 << 20))
    assert set(other) <= set(a)
    a.update(other)
    head = (a["q"],) if call != "append" else (a["q"], a["k"], a["v"])
    tail = (a["workspace"],) if call != "noalloc" else ()
    fn = {"decode": pa.pa_decode, "append": pa.pa_append_decode, "noalloc": pa.pa_decode_noalloc}[call]
    fn(*head, a["k_cache"], a["v_cache"], a["tables"], a["lens"], 32, 0.125, a["out"], *tail, DESC, opts, stream=0)


BAD = [
    ("q", Fake(torch.bfloat16, ROWS - 1), "needs"),
    ("q", Fake(torch.bfloat16, ROWS, device=1), "current device"),
    ("out", Fake(torch.bfloat16, ROWS - 1), "needs"),
    ("out", Fake(torch.bfloat16, ROWS, device=1), "current device"),
    ("k_cache", Fake(torch.uint8, POOL * 9 // 16, device=1), "current device"),
    ("v_cache", Fake(torch.uint8, POOL * 9 // 16 - 1), "needs"),
    ("tables", Fake(torch.int32, 5), "needs"),
    ("tables", Fake(torch.int32, 6, device=1), "current device"),
    ("lens", Fake(torch.int32, 3, device=1), "current device"),
    ("lens", Fake(torch.int32, 3, device=-1), "CUDA"),
]


@pytest.mark.parametrize("name,tensor,text", BAD)
@pytest.mark.parametrize("call", ["decode", "append", "noalloc"])
def test_decode(library, call, name, tensor, text):
    with pytest.raises(ValueError, match=text):
        decode(call, **{name: tensor})
    assert not library


@pytest.mark.parametrize("call", ["decode", "append"])
@pytest.mark.parametrize("tensor,text", [(Space(torch.uint8, 1 << 20, device=1), "current device"),
                                         (Space(torch.uint8, 1 << 20, device=-1), "current device"),
                                         (Space(torch.uint8, 1 << 20, contiguous=False), "contiguous")])
def test_decode_workspaces(library, call, tensor, text):
    with pytest.raises(ValueError, match=text):
        decode(call, workspace=tensor)
    assert not library


@pytest.mark.parametrize("name,tensor,text", [("k", Fake(torch.bfloat16, NEW - 1), "needs"),
                                              ("v", Fake(torch.bfloat16, NEW, device=1), "current device")])
def test_new_rows(library, name, tensor, text):
    with pytest.raises(ValueError, match=text):
        decode("append", **{name: tensor})
    assert not library


def test_calls_that_pass(library):
    for call in ("decode", "append", "noalloc"):
        decode(call)
        decode(call, opts=None)
        decode(call, q=4096, out=4096, tables=4096)        # raw addresses
    decode("decode", workspace=Space(torch.float32, 1 << 18))
    assert len(library) == 10


@pytest.mark.parametrize("call", ["prefill", "cross"])
def test_output_as_long_as_the_rows(library, call):
    fn = pa.pa_prefill_ex if call == "prefill" else pa.pa_cross_attention
    rest = (Fake(torch.bfloat16, POOL), Fake(torch.bfloat16, POOL), Fake(torch.int32, 6), Fake(torch.int32, 4),
            Fake(torch.int32, 3), 4, 32, 0.125)
    ws = Fake(torch.uint8, 1 << 20)
    with pytest.raises(ValueError, match="needs"):
        fn(Fake(torch.bfloat16, ROWS), *rest, Fake(torch.bfloat16, ROWS - 1), ws, DESC, stream=0)
    assert not library
    fn(Fake(torch.bfloat16, ROWS), *rest, Fake(torch.bfloat16, ROWS), ws, DESC, stream=0)
    fn(4096, *rest, Fake(torch.bfloat16, 1), ws, DESC, stream=0)
    assert len(library) == 2
