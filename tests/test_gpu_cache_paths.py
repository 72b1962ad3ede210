"""Paths of the paged-cache operators that the sizes of test_gpu_cache.py leave
out, against the same oracle and with its bounds."""
import pytest

import test_gpu_cache as t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,n,dim", [(1, 40000, 64), (3, 12000, 128),
                                         (5, 9000, 256), (15, 4001, 64)])
def test_attend_long_rows_of_odd_groups(group, n, dim):
    """Joined by the second launch, from shares of an odd number of queries."""
    rng, dev, ref = t._case(group, [n, n // 3], 1, dim, 16, "bf16")
    print("attend odd group", group, n, dim, flush=True)
    t._attend(dev, t._q(rng, 2, group, dim, "bf16"), ref, "bf16", "bf16",
              rng=rng)


@pytest.mark.parametrize("lens,keep,extra", [
    ([2000, 0, 1, 1024], 2000, 80), ([500, 20000, 3000, 4096], 4096, 1),
    ([100, 90], 64, 80)])
@pytest.mark.parametrize("kind", ["plain", "special"])
def test_evict_short_rows_in_a_wide_table(lens, keep, extra, kind):
    """Rows of at most `keep` slots, and short rows that are cut, where the
    table can name more slots than one workgroup selects from."""
    print("evict in a wide table", lens, keep, kind, flush=True)
    t._check_evict(lens, 2, 8, 256, keep, 4, 20, kind, extra=extra)
