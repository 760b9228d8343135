"""What mla_pages_reserve reports when the pool is too small: the pages missing, also where one sequence alone asks for
more than the pool has."""
import pytest

from tests.test_decode_pages_gpu import Both

pytestmark = pytest.mark.gpu


def test_one_request_larger_than_the_pool():
    b = Both(10, 4, 5, 30)
    assert b.reserve([0], [100]) == 15             # 25 pages wanted, 10 free
    assert b.reserve([0, 1], [9, 100]) == 18       # 3 + 25
    assert b.reserve([0], [9]) == 0
    assert b.reserve([0, 1, 2], [120, 50, 44]) == 44   # 27 + 13 + 11, 7 free
    b.set_lens([9, 0, 0, 0, 0])
    b.fork([0], [1])
    assert b.reserve([1, 2], [40, 60]) == 19       # a copy, 10 and 15 pages, 7 free
    assert b.reserve([1], [8]) == 0


def test_many_requests_larger_than_the_pool():
    b = Both(6, 1, 300, 5000)
    n = 300
    assert b.reserve(list(range(n)), [5000 - k for k in range(n)]) == sum(5000 - k for k in range(n)) - 6
    assert b.reserve([7, 7, 9, -1], [3, 900, 4000, 8]) == 3997
