"""Block-scaled and mixture-of-experts entry points, host side: what a call hands to the library is made from the
tensors as they are at that call, whatever other threads do.  Nothing here launches a kernel."""
import ctypes
import threading

import pytest
import torch

from hpc_linear_algebra_amd import blocks

E4 = torch.float8_e4m3fn


def made(rows=4, k=40):
    return blocks._made(torch.zeros(rows, 48, dtype=E4), torch.ones(1, rows), rows, k, 1)


class Recorder:
    """Stands for the extension module: keeps what its product was called with."""

    def __init__(self):
        self.calls = []

    def gemm(self, *args):
        self.calls.append(args)
        return torch.zeros(0)


def test_threads_that_first_multiply_one_matrix_share_no_descriptor(monkeypatch):
    """Two threads enter the first product of a matrix together: nothing that one of them hands over may be an address
    inside an object which the other has replaced."""
    blocks.T.lib()
    both = threading.Barrier(2)
    struct = blocks.T.tlr_block_matrix

    def slow(*args):
        try:
            both.wait(2)                     # both threads have seen that there is none yet
        except threading.BrokenBarrierError:
            pass
        return struct(*args)

    rec = Recorder()
    monkeypatch.setattr(blocks.T, "tlr_block_matrix", slow)
    monkeypatch.setattr(blocks, "binding", lambda: rec)
    q = made()
    threads = [threading.Thread(target=blocks.gemm, args=(q, q)) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(rec.calls) == 2
    alive = ctypes.addressof(q._c) if getattr(q, "_c", None) is not None else None
    for args in rec.calls:
        for a in args[:2]:
            assert isinstance(a, torch.Tensor) or a == alive


def test_descriptor_follows_its_tensors():
    q = made()
    assert (q.c.codes, q.c.scales, q.c.ld) == (q.codes.data_ptr(), q.scales.data_ptr(), 48)
    first = q.codes                                  # alive, so that the addresses differ
    q.codes, q.scales = torch.zeros(4, 64, dtype=E4), torch.ones(1, 8)[:, :4]
    assert (q.c.codes, q.c.scales, q.c.ld) == (q.codes.data_ptr(), q.scales.data_ptr(), 64)
    assert q.c.codes != first.data_ptr()
    p = blocks.BlockScaled(torch.zeros(4, 48, dtype=E4), torch.ones(1, 4), 4, 40, 1)
    p.codes = torch.zeros(4, 80, dtype=E4)
    assert (p.c.codes, p.c.ld) == (p.codes.data_ptr(), 80)


@pytest.mark.parametrize("codes,scales", [
    (torch.zeros(3, 48, dtype=E4), torch.ones(1, 4)), (torch.zeros(4, 32, dtype=E4), torch.ones(1, 4)),
    (torch.zeros(4, 48), torch.ones(1, 4)), (torch.zeros(4, 48, dtype=E4), torch.ones(1, 3)),
    (torch.zeros(4, 48, dtype=E4), torch.ones(1, 4, dtype=torch.float64)),
    (torch.zeros(4, 48, dtype=E4), torch.ones(4, 2)[:, :1].t()),
    (torch.zeros(48, 4, dtype=E4).t(), torch.ones(1, 4)), (torch.zeros(4, 40, dtype=E4), torch.ones(1, 4))])
def test_a_replaced_tensor_that_does_not_fit_is_refused(codes, scales):
    """The product checks the tensors that it is given, not those that the matrix was made with."""
    q = made()
    q.codes, q.scales = codes, scales
    with pytest.raises(ValueError):
        q.c
    with pytest.raises(ValueError):
        blocks.gemm(q, made())


def test_a_layer_hands_out_nothing_that_its_calls_point_into():
    from hpc_linear_algebra_amd import moe
    layer = moe.MoELayer.__new__(moe.MoELayer)
    for name in ("c", "ws"):
        with pytest.raises(AttributeError):
            setattr(layer, name, torch.zeros(1))
    layer._c = blocks.T.tlr_moe_layer(64, 32, 8, 2)
    layer.c.hidden = 1 << 20
    assert layer.c.hidden == 64 and ctypes.addressof(layer.c) != ctypes.addressof(layer._c)


def test_a_layer_refuses_what_requires_a_gradient():
    from hpc_linear_algebra_amd import moe
    layer = moe.MoELayer.__new__(moe.MoELayer)
    layer.device, layer._trained = torch.device("cuda", 0), False
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="no backward"):
        layer(x.requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError):             # x is not on the layer's device
        layer(x)
    layer._trained = True
    with pytest.raises(RuntimeError, match="no backward"):
        layer(x.detach())


def test_an_unknown_result_type_is_an_argument_error():
    q = made()
    for bad in ("f64", "e4m3", "float32", None, 3):
        with pytest.raises(ValueError, match="dtype"):
            blocks.gemm(q, q, dtype=bad)
