"""The binding's compiled module next to Python: errors of Python objects."""
import pytest
import torch

PARAM = 5


class NoTruth:
    def __bool__(self):
        raise ValueError("neither true nor false")


@pytest.fixture(scope="module")
def m():
    import speculative_decoding_logit_gb300 as asv
    asv.build()
    from speculative_decoding_logit_gb300 import _binding
    return _binding


def test_interleaved_without_a_truth_value_is_refused(m):
    """Before anything else is looked at."""
    x = torch.zeros(1)
    with pytest.raises(m.AsvError) as e:
        m._paged_ext().paged_kv_append(x, x, x, x, x, x, x, None, None, NoTruth(), None, x, 0)
    assert e.value.status == PARAM


def _small_call():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c, q = torch.zeros(2, 16, 2, 64, **bf), torch.zeros(1, 4, 64, **bf)
    return c, q, torch.zeros(1, 1, **i32), torch.zeros(1, **i32), torch.tensor([0, 1], **i32)


@pytest.mark.gpu
def test_interleaved_of_a_whole_call(m):
    c, q, table, length, indptr = _small_call()
    rot = torch.zeros(4, 64, device="cuda")
    before = c.clone()
    c2 = c.clone()
    with pytest.raises(m.AsvError) as e:
        m.paged_kv_append(q[:, :2] + 1, q[:, :2] + 1, c, c2, table, length, indptr, rotary=rot, interleaved=NoTruth())
    assert e.value.status == PARAM and torch.equal(c, before) and torch.equal(c2, before)
    m.paged_kv_append(q[:, :2], q[:, :2], c, c2, table, length, indptr, rotary=rot, interleaved=1)
