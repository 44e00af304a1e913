"""What the binding refuses before a call reaches the library: tensors of another device than the
current one, of another type, too small for the pool, the tables or the rows that the call names."""
import pytest
import torch

import pagedattention_kv_cache_pa_b200 as pa
from pagedattention_kv_cache_pa_b200 import binding

DESC = pa.CacheDesc.make(num_blocks=4, block_size=16, num_kv_heads=2, num_q_heads=4, head_dim=64,
                         max_blocks_per_seq=2)
POOL = 4 * 2 * 16 * 64


class Fake:
    """A tensor as the checks see one; nothing reads its address."""
    def __init__(self, dtype, n, device=0, contiguous=True, rows=None):
        self.dtype, self.n, self.index, self.contiguous = dtype, n, device, contiguous
        self.shape = (n if rows is None else rows,)
        self.device = "cuda:%d" % device if device >= 0 else "cpu"

    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.n

    def data_ptr(self):
        return 256


@pytest.fixture(autouse=True)
def device_zero(monkeypatch):
    monkeypatch.setattr(binding, "_device", lambda: 0)


def append_args(**other):
    a = dict(k=Fake(torch.bfloat16, 3 * 2 * 64), v=Fake(torch.bfloat16, 3 * 2 * 64), slots=Fake(torch.int64, 3),
             k_cache=Fake(torch.uint8, POOL * 9 // 16), v_cache=Fake(torch.uint8, POOL * 9 // 16))
    a.update(other)
    return a


@pytest.mark.parametrize("name,tensor,error,text", [
    ("k", Fake(torch.bfloat16, 3 * 2 * 64, device=1), ValueError, "current device"),
    ("slots", Fake(torch.int64, 3, device=1), ValueError, "current device"),
    ("v_cache", Fake(torch.uint8, POOL * 9 // 16, device=1), ValueError, "current device"),
    ("v", Fake(torch.bfloat16, 3 * 2 * 64, device=-1), ValueError, "CUDA"),
    ("v", Fake(torch.float16, 3 * 2 * 64), TypeError, "bfloat16"),
    ("v", Fake(torch.bfloat16, 3 * 2 * 64 - 1), ValueError, "needs"),
    ("k", Fake(torch.bfloat16, 3 * 2 * 64, contiguous=False), ValueError, "contiguous"),
    ("k_cache", Fake(torch.uint8, POOL * 9 // 16 - 1), ValueError, "needs"),
    ("k_cache", Fake(torch.bfloat16, POOL), TypeError, "uint8"),
])
@pytest.mark.parametrize("call", ["append", "gather"])
def test_rows_and_pools(call, name, tensor, error, text):
    a = append_args(**{name: tensor})
    with pytest.raises(error, match=text):
        if call == "append":
            pa.pa_append_kv_e2m1(a["k"], a["v"], a["slots"], 1.0, 1.0, a["k_cache"], a["v_cache"], DESC, stream=0)
        else:
            pa.pa_gather_kv_e2m1(a["k_cache"], a["v_cache"], a["slots"], 1.0, 1.0, a["k"], a["v"], DESC, stream=0)


ROWS = 3 * 4 * 64


@pytest.mark.parametrize("name,tensor,text", [
    ("q", Fake(torch.bfloat16, ROWS, device=1), "current device"),
    ("out", Fake(torch.bfloat16, ROWS, device=1), "current device"),
    ("k_cache", Fake(torch.bfloat16, POOL, device=1), "current device"),
    ("v_cache", Fake(torch.bfloat16, POOL - 1), "needs"),
    ("tables", Fake(torch.int32, 5), "needs"),
    ("cu", Fake(torch.int32, 3), "needs"),
    ("lens", Fake(torch.int32, 3, device=1), "current device"),
    ("workspace", Fake(torch.uint8, 1 << 20, device=1), "current device"),
])
@pytest.mark.parametrize("call", ["prefill", "cross"])
def test_attention(call, name, tensor, text):
    a = dict(q=Fake(torch.bfloat16, ROWS), out=Fake(torch.bfloat16, ROWS), k_cache=Fake(torch.bfloat16, POOL),
             v_cache=Fake(torch.bfloat16, POOL), tables=Fake(torch.int32, 6), cu=Fake(torch.int32, 4),
             lens=Fake(torch.int32, 3), workspace=Fake(torch.uint8, 1 << 20))
    a[name] = tensor
    fn = pa.pa_prefill_ex if call == "prefill" else pa.pa_cross_attention
    with pytest.raises(ValueError, match=text):
        fn(a["q"], a["k_cache"], a["v_cache"], a["tables"], a["cu"], a["lens"], 4, 32, 0.125, a["out"],
           a["workspace"], DESC, stream=0)


def test_cross_of_one_row_a_sequence_checks_its_rows():
    with pytest.raises(ValueError, match="needs"):
        pa.pa_cross_attention(Fake(torch.bfloat16, ROWS - 1), Fake(torch.bfloat16, POOL), Fake(torch.bfloat16, POOL),
                              Fake(torch.int32, 6), None, Fake(torch.int32, 3), 1, 32, 0.125,
                              Fake(torch.bfloat16, ROWS), Fake(torch.uint8, 1 << 20), DESC, stream=0)
