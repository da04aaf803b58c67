"""The binding's native checks of tensor arguments (csrc/host_args.cpp): what they take is
what the checks in Python take, and what they do not take is refused with the same words."""
import pytest
import torch

from linear_attention_serving_gated_gb300 import kda


@pytest.fixture(scope="module")
def host():
    kda.load()
    from linear_attention_serving_gated_gb300 import _host_args

    assert kda._arg is _host_args.arg and kda._rows is _host_args.rows and kda._states is _host_args.states
    return _host_args


class Odd:
    dtype = torch.float32


def test_refusals_are_those_of_the_python_checks(host):
    x = torch.zeros(4, 8)
    cases = [(x, torch.float32, 0), (x, torch.bfloat16, 0), (x.t(), torch.float32, 0), (x, torch.float32, 33), (Odd(), torch.float32, 0),
             (None, torch.float32, 0), (x, torch.float32, 2 ** 70), (torch.empty(4, 8, device="meta"), torch.float32, 0)]
    for t, dtype, n in cases:
        said = []
        for check in (host.arg, kda._checked_arg):
            with pytest.raises(Exception) as e:
                check(t, dtype, n, "x", "[n]")
            said.append((type(e.value), str(e.value)))
        assert said[0] == said[1]


def test_no_rows_and_no_states(host):
    x = torch.zeros(4, 8)
    for args in ((x, torch.float32, 4, 8), (None, torch.float32, 4, 8), (x, "float32", 4, 8), (x, torch.float32, None, 8), (x,), ()):
        assert host.rows(*args) is None
    p = torch.zeros(2, 3, 4, 5)
    for args in ((p, 3, 4, 5), (None, 3, 4, 5), (p, 3, 4, "5"), (p, 2 ** 70, 4, 5), ()):
        assert host.states(*args) is None


@pytest.mark.gpu
def test_pointers(host):
    x = torch.zeros(6, 8, dtype=torch.bfloat16, device="cuda")
    for t, dtype in ((x, torch.bfloat16), (x[2:], torch.bfloat16), (x.view(torch.int16), torch.float16), (x[:0], torch.bfloat16),
                     (torch.nn.Parameter(x), torch.bfloat16)):
        assert host.arg(t, dtype, t.numel(), "x", "[n]") == t.data_ptr() == kda._checked_arg(t, dtype, t.numel(), "x", "[n]")
    for t, dtype, n in ((x, torch.float16, 0), (x[:, 1:], torch.bfloat16, 0), (x, torch.bfloat16, 49), (x.float(), torch.bfloat16, 0)):
        with pytest.raises((TypeError, ValueError)):
            host.arg(t, dtype, n, "x", "[n]")
    assert host.rows(x[1:, 2:], torch.bfloat16, 5, 6) == (x[1:, 2:].data_ptr(), 8)
    for t, dtype, n, width in ((x, torch.float16, 6, 8), (x, torch.bfloat16, 7, 8), (x, torch.bfloat16, 6, 9), (x.t(), torch.bfloat16, 6, 6),
                               (x[0], torch.bfloat16, 1, 8)):
        assert host.rows(t, dtype, n, width) is None
    p = torch.zeros(3, 2, 4, 5, device="cuda")
    assert host.states(p, 2, 4, 5) == (p.data_ptr(), 3) and host.states(p[:0], 2, 4, 5)[1] == 0
    for t, sizes in ((p, (2, 5, 4)), (p.transpose(2, 3), (2, 5, 4)), (p.half(), (2, 4, 5)), (p[0], (2, 4, 5)), (p[:, :1], (1, 4, 5))):
        assert host.states(t, *sizes) is None
