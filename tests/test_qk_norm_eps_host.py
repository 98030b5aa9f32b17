"""The range of eps of the head norms (no GPU needed): a subnormal one, with which a zero head would be 0 times infinity, is refused."""
import pytest

from test_qk_norm_host import _backward, _forward

FLT_MIN = 2.0 ** -126


@pytest.mark.parametrize("f", [_forward, _backward])
def test_subnormal_eps_is_refused(f):
    more = {"T": 0, **({} if f is _forward else dict(dgq=None, dgk=None))}          # nothing is enqueued where it is accepted
    for eps in (2.0 ** -149, 1e-40, FLT_MIN - 2.0 ** -149):
        assert f(eps=eps, **more) == 4, eps
        assert f(eps=eps, gq=None, gk=None, **more) == 0, eps             # without a norm eps is ignored
    for eps in (FLT_MIN, 1e-37, 1e-6, 2.9e38):
        assert f(eps=eps, **more) == 0, eps
