"""The table of axes that spc_norm_rope hands to the library, from every kind of sequence that it may be given as."""
import array
import ctypes as C

import numpy as np
import pytest
import torch

import bit_kv_cache_spc_gb300 as spc

ROT, AXES = 48, 3
TABLE = [i % AXES for i in range(ROT // 2)]


@pytest.fixture
def packed(monkeypatch):
    """A call on host tensors, marshalled and not made: the table in its dims."""
    rows = (0, (1, 2, 4, 2, 128), (0,) * 18, (None,) * 6)
    monkeypatch.setattr(spc, "_rope_rows", lambda *_: rows)
    monkeypatch.setattr(spc, "_words", lambda *_: None)
    monkeypatch.setattr(spc, "_raw_stream", lambda *_: None)

    def table(axis, pos=torch.zeros((AXES, 1, 2), dtype=torch.int32)):
        later = []
        spc.spc_norm_rope(None, None, pos, None, axis=axis, rot=ROT, _later=later)
        d = spc.spc_norm_rope_dims.from_buffer_copy(later[0][1][0])
        assert d.axes == AXES
        return list(d.axis)

    return table


@pytest.mark.parametrize("kind", [
    list, tuple, bytes, bytearray, np.array, lambda x: np.array(x, dtype=np.int32), lambda x: np.array(x, dtype=np.uint8),
    lambda x: np.array(x, dtype=np.int16)[::-1][::-1], lambda x: array.array("i", x), lambda x: array.array("B", x),
    lambda x: memoryview(array.array("q", x)), lambda x: (C.c_int32 * len(x))(*x), torch.tensor,
    lambda x: [np.int64(a) for a in x]])
def test_entry_by_entry(packed, kind):
    assert packed(kind(TABLE)) == TABLE + [0] * (64 - len(TABLE))


@pytest.mark.parametrize("bad", [
    TABLE[:-1], TABLE + [0], [], np.array(TABLE[:-1]), np.array(TABLE + [0] * 168), bytes(8 * len(TABLE)), [256] * len(TABLE),
    [-1] * len(TABLE), np.full(len(TABLE), -1), None])
def test_other_numbers_are_refused(packed, bad):
    with pytest.raises(ValueError):
        packed(bad)


@pytest.mark.parametrize("bad", [[0.0] * len(TABLE), np.zeros(len(TABLE)), "0" * len(TABLE), 5])
def test_what_holds_no_whole_numbers_is_refused(packed, bad):
    with pytest.raises(TypeError):
        packed(bad)


@pytest.mark.parametrize("shape", [(1, 2, AXES), (AXES, 2, 1), (AXES, 1, 3), (AXES, 2, 2)])
def test_positions_of_another_order_are_refused(packed, shape):
    """One sequence of two tokens: [axes][1][2] alone."""
    with pytest.raises(ValueError):
        packed(TABLE, torch.zeros(shape, dtype=torch.int32))


def test_as_many_axes_as_sequences(monkeypatch, packed):
    """[B][T][axes] has then the shape's first number and its count of elements right."""
    monkeypatch.setattr(spc, "_rope_rows", lambda *_: (0, (AXES, 7, 4, 2, 128), (0,) * 18, (None,) * 6))
    with pytest.raises(ValueError):
        packed(TABLE, torch.zeros((AXES, 7, AXES), dtype=torch.int32))
    assert packed(TABLE, torch.zeros((AXES, AXES, 7), dtype=torch.int32))[:3] == TABLE[:3]
