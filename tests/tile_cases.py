"""Sizes that reach each tile of the cross entropy's and the MXFP8 weight
gradient's products, whole and in parts of K, on 256 compute units:
{(rows, columns, in parts): cases}."""

# T, V, D of the logits
LOGITS = {(64, 128, False): [(64, 70001, 64), (130, 1000, 200), (1025, 769, 1032)],
          (128, 128, False): [(100, 40001, 64), (128, 33000, 72)],
          (192, 256, False): [(333, 50021, 64), (513, 25700, 72)],
          (256, 256, False): [(256, 65536, 64), (250, 65500, 136)]}
# T, V, D of dh, contracted over V
DH = {(64, 128, False): [(300, 200, 520)], (64, 128, True): [(37, 8191, 1032), (64, 70001, 64)],
      (128, 128, False): [(2000, 200, 2048)], (128, 128, True): [(1000, 3000, 1024), (513, 25700, 136)],
      (192, 256, False): [(3000, 136, 4096)], (192, 256, True): [(800, 12000, 2056)],
      (256, 256, False): [(4096, 256, 4096)], (256, 256, True): [(4352, 4099, 4096)]}
# T, V, D of dw, contracted over T
DW = {(128, 128, False): [(300, 2000, 2000)], (128, 128, True): [(8192, 1000, 512), (2000, 3000, 2048)],
      (256, 256, False): [(37, 8191, 1032), (130, 70001, 264)], (256, 256, True): [(1100, 4351, 4096)]}
# T, Din, Dout
WGRAD = {(128, 128, False): [(300, 96, 1032)], (128, 128, True): [(4100, 288, 264), (1000, 224, 520)],
         (256, 256, False): [(70, 8224, 2056), (330, 4128, 4616)],
         (256, 256, True): [(2000, 2048, 3000), (1100, 4096, 4352)]}


def flat(table):
    return [c for cases in table.values() for c in cases]
