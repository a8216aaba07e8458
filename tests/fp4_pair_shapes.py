"""Products that CTA pairs multiply, with last tiles of tokens and of weight rows that are not full: (tokens, weight rows,
columns, weight rows to a tile on a GPU of 152 SMs). N is a multiple of 8, as the pairs' stores need it, but of no tile."""

SHAPES = [(24, 520, 512, 128), (130, 296, 640, 128), (150, 2056, 1408, 128), (200, 328, 512, 128),
          (700, 3336, 640, 256), (1200, 2056, 512, 256), (2049, 1032, 640, 256),
          (600, 7000, 2176, 384), (769, 6920, 2176, 384)]
