"""The protocol model of the tree-attention kernel at the rings that it is built
with (two stages of K and V at D = 128, four at D = 64, one row block or two), and
the ring of the key masks: K's producer writes a tile's masks when it starts the
tile, up to STAGES + 1 tiles ahead, and the MMA warp and the softmax rows read
them before the tile's P V."""
import random

import pytest

from test_cache_protocol_cpu import Model, Overtaken, pieces_of

OK_RING = 8  # tiles whose masks are kept


class Copies(list):
    """The copies in flight; a tile of K notes its masks as it is started."""

    def __init__(self, model):
        super().__init__()
        self.model = model

    def append(self, copy):
        if copy[1] == "k":
            self.model.masks[copy[3] % self.model.ring] = copy[3]
        super().append(copy)


class Masks(Model):
    def __init__(self, *args, ring=OK_RING, **kw):
        super().__init__(*args, **kw)
        self.ring, self.masks = ring, {}
        self.copies = Copies(self)

    def step_async(self):
        # P V of a tile runs behind every read of its masks: what holds then held for them
        if self.pipe and self.pipe[0][0] == "pv":
            at = self.pipe[0][3]
            assert self.masks[at % self.ring] == at, "masks of another tile"
        return super().step_async()


@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("NT,stages", [(1, 2), (1, 4), (2, 2), (2, 4)])
def test_built_rings_are_sound(NT, stages, rows):
    for seed in range(150):
        rng = random.Random(seed * 29 + NT * 5 + stages)
        Masks(NT, stages, stages, pieces_of(rng), rng, rows=rows).run()


@pytest.mark.parametrize("stages", [2, 4])
def test_one_barrier_for_two_score_buffers_is_found(stages):
    found = 0
    for seed in range(300):
        rng = random.Random(seed)
        try:
            Masks(1, stages, stages, pieces_of(rng), rng, shared_p=True).run()
        except Overtaken:
            found += 1
    assert found


def test_a_ring_of_masks_that_is_too_short_is_found():
    found = 0
    for seed in range(100):
        rng = random.Random(seed)
        try:
            Masks(1, 4, 4, pieces_of(rng), rng, ring=4).run()
        except AssertionError as e:
            found += "masks of another tile" in str(e)
    assert found
