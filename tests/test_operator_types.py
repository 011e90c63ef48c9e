"""Element types in the operators' binding: a tensor of another type than the
call reads or writes has bytes enough (int64 ids, a float64 bias) or the same
number of them (float16 for bfloat16), and is refused.  On the CPU: the tensors
only say that they lie on a device, and nothing is called."""
import pytest
import torch

import quantized_linear_layer_amd as qll

F, D, H, B, I, L = torch.float32, torch.float64, torch.float16, torch.bfloat16, torch.int32, torch.int64


class OnDevice:
    def __init__(self, dtype, n=4096):
        self.dtype, self.nbytes = dtype, n * torch.empty(0, dtype=dtype).element_size()

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def taken(monkeypatch):
    """What reaches the library, in place of the call."""
    calls = []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(qll, "_raw_stream", None)
    monkeypatch.setattr(qll, "_current_device", None)
    monkeypatch.setattr(qll, "_call", lambda name, *args: calls.append(name))
    return calls


def t(dtype):
    return OnDevice(dtype)


U = torch.uint8
CALLS = {  # entry: arguments, and by position of a typed one the types that it refuses
    "qll_rmsnorm_q8_0": ([t(B), qll.QLL_DTYPE_BF16, t(B), t(F), 1e-5, t(B), t(U), 2, 64],
                         {0: (H, F), 2: (H, F), 3: (D,), 5: (H, F)}),
    "qll_rmsnorm_i8_rows": ([t(H), qll.QLL_DTYPE_F16, t(H), t(F), 1e-5, t(H), t(torch.int8), t(F), t(I), 2, 64],
                            {0: (B, F), 2: (B, D), 3: (D,), 5: (B,), 7: (D, I), 8: (L, F)}),
    "qll_q4_0_q8_0_linear": ([t(U), t(U), t(F), 0, t(F), t(F), 2, 8, 32], {2: (D, B), 4: (D, I), 5: (D, B)}),
    "qll_q4_0_repacked_q8_0_linear": ([t(U), t(U), t(F), 0, t(F), t(F), 2, 8, 32], {2: (D,), 4: (D,), 5: (D, L)}),
    "qll_q4_0_q8_0_gated": ([t(U), t(U), t(U), 0, t(F), 2, 8, 32], {4: (D, B)}),
    "qll_q4_0_repacked_q8_0_gated": ([t(U), t(U), 0, t(F), 2, 8, 32], {3: (D, B)}),
    "qll_token_logprobs": ([t(F), qll.QLL_DTYPE_F32, t(I), 2, t(F), t(F), 3, t(I), t(F), 4, 100],
                           {0: (D, I), 2: (L, F), 4: (D,), 5: (D,), 7: (L, F), 8: (D,)}),
}


@pytest.mark.parametrize("name", CALLS)
def test_other_types_are_refused(taken, name, monkeypatch):
    monkeypatch.setattr(qll, "_repacked_need", lambda n, k, gated: 1)
    args, bad = CALLS[name]
    getattr(qll, name)(*args)
    assert taken == [name]
    for at, types in bad.items():
        for dtype in types:
            a = list(args)
            a[at] = t(dtype)
            with pytest.raises(ValueError, match="is of type"):
                getattr(qll, name)(*a)
    assert taken == [name]


def test_ids_of_torchs_default_type(taken):
    """The natural mistake: ids as torch makes them."""
    with pytest.raises(ValueError, match="tokens is of type torch.int64, the call takes torch.int32"):
        qll.qll_token_logprobs(t(F), 0, OnDevice(torch.tensor([1, 2]).dtype), 1, t(F), None, 0, None, None, 2, 100)


def test_raw_bits_parts_left_out_and_unknown_types(taken):
    qll.qll_token_logprobs(t(torch.int16), qll.QLL_DTYPE_BF16, None, 0, None, None, 0, None, None, 2, 100)
    qll.qll_token_logprobs(t(U), qll.QLL_DTYPE_F16, t(L), 0, t(D), None, 0, t(L), t(D), 2, 100)  # t and top are 0
    qll.qll_token_logprobs(t(U), 7, None, 0, None, None, 0, None, None, 2, 100)  # the library's to refuse
    assert len(taken) == 3
