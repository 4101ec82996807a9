"""The binding of the 4-bit cache without a GPU: sizes that a C int does not hold, against a library that records its
arguments and tensors that have a shape and an address only; and a torch without the private names that it shortens
the way with."""
import numpy as np
import pytest
import torch

import alibi_positional_bias_gb300 as ab

BIG = 2 ** 32


class Tensor:
    """What the binding asks of a tensor on cuda:0."""

    def __init__(self, *shape, dtype=torch.bfloat16):
        self.shape, self.dtype = shape, dtype

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Library:
    """Takes its arguments as C ints, as ctypes hands them over, and records them."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(tuple(int(np.array(a, dtype=np.int64).astype(np.int32)) if isinstance(a, int) and i > 4 else a
                                    for i, a in enumerate(args)))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = Library()
    monkeypatch.setattr(ab, "_names", (torch.bfloat16, torch.uint8, torch.int32, torch.float32, lambda index: 0, lambda: 0, fake))
    return fake


def decode(L, blocks=2):
    q = Tensor(1, 2, 1, 64)
    return ab.alibi_attn_decode_kv4(q, Tensor(1, 2, blocks, 2304, dtype=torch.uint8), L=L, out=Tensor(1, 2, 1, 64),
                                    lse=Tensor(1, 2, 1, dtype=torch.float32))


def test_decode_passes_the_bound_on(lib):
    for L in (1, 33, 64, None):
        decode(L)
        assert lib.calls[-1][5:12] == (1, 2, 2, 1, 64 if L is None else L, 64, 64)


@pytest.mark.parametrize("L", [0, -1, 65, BIG + 1, BIG + 64, -BIG + 64, 2 ** 31, 2 ** 63])
def test_decode_refuses_a_bound_beyond_the_capacity(lib, L):
    with pytest.raises(ab.AlibiError) as e:
        decode(L)
    assert e.value.status == ab.ALIBI_ERR_INVALID and not lib.calls


@pytest.mark.parametrize("tokens", [(1 << 24) + 32, 2 ** 31, BIG + 32])
def test_capacities_beyond_the_largest_are_refused(lib, tokens):
    k, c = Tensor(1, 2, 1, 64), Tensor(1, 2, tokens // 32, 2304, dtype=torch.uint8)
    for call in (lambda: decode(32, tokens // 32), lambda: ab.alibi_kv4_write(k, k, c), lambda: ab.alibi_kv4_read(c, k, k)):
        with pytest.raises(ab.AlibiError) as e:
            call()
        assert e.value.status == ab.ALIBI_ERR_UNSUPPORTED and not lib.calls


@pytest.mark.parametrize("T", [0, 65, 2 ** 31, BIG + 1])
def test_more_tokens_than_the_capacity_are_refused(lib, T):
    k, c = Tensor(1, 2, T, 64), Tensor(1, 2, 2, 2304, dtype=torch.uint8)
    for call in (lambda: ab.alibi_kv4_write(k, k, c), lambda: ab.alibi_kv4_read(c, k, k)):
        with pytest.raises(ab.AlibiError) as e:
            call()
        assert e.value.status == ab.ALIBI_ERR_INVALID and not lib.calls
    k = Tensor(1, 2, 64, 64)
    ab.alibi_kv4_write(k, k, c)
    assert lib.calls[-1][5:10] == (1, 2, 64, 64, 64)


def test_head_sizes_that_no_int_holds():
    for d in (BIG + 64, 2 ** 31, -BIG + 64):
        with pytest.raises(ab.AlibiError):
            ab.alibi_kv4_block_bytes(d)


def test_a_torch_without_its_private_shortcuts(monkeypatch):
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)

    class Stream:
        cuda_stream = 77
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream if index == 1 else None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(ab, "load", lambda: "library")
    monkeypatch.setattr(ab, "_names", None)
    names = ab._kv4_names()
    assert names[4](1) == 77 and names[5]() == 1 and names[6] == "library"
