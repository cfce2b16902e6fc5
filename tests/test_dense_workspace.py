"""The workspace of the linear layer's backward pass: as the header says, every call wants it, whichever gradients it asks for
(fake aligned addresses, with an injected launch failure behind the checks: nothing is dereferenced)."""
import os
import re

import pytest

from tests.test_dense_refusals import ARG, CUDA, lib, linear_backward, no_launch  # noqa: F401

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "linattn.h")


@pytest.mark.parametrize("act", [0, 1, 4])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (4, 8, 64), (10, 60, 70), (5000, 60, 70), (40, 60, 72)])
def test_every_call_wants_it(lib, m, n, k, act):  # noqa: F811
    need = lib._load().la_linear_backward_workspace_bytes(m, n, k, act)
    assert need > 0
    whole = lambda c: (c + 7) // 8 * 8  # noqa: E731
    sizes = dict(M=m, N=n, K=k, act=act, sb=2 ** 40, ldx=whole(k), ldw=whole(k), lddx=whole(k), lddw=whole(k), lddy=whole(n))
    for asked in ({}, dict(dx=None, dbias=None), dict(dw=None, dbias=None), dict(dx=None, dw=None)):
        assert linear_backward(lib, **sizes, **asked, wsb=need) == CUDA
        assert linear_backward(lib, **sizes, **asked, wsb=need - 1) == ARG and "workspace" in lib.last_error()
        assert linear_backward(lib, **sizes, **asked, ws=None, wsb=0) == ARG and "workspace" in lib.last_error()


def test_the_header_offers_no_call_without_it():
    text = open(HEADER).read()
    at = text.index("size_t la_linear_backward_workspace_bytes")
    said = re.sub(r"\s*\n \*\s*", " ", text[text.rindex("/*", 0, at):at])
    assert "never 0" in said and "may be NULL when" not in said
