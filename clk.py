import torch,ctypes,sys
sys.path.insert(0,'.')
from linear_latent_routing_gb300 import attention as A, gma
q,k,v=torch.randn(1,8192,16,128,device='cuda').bfloat16(),torch.randn(1,8192,4,128,device='cuda').bfloat16(),torch.randn(1,8192,4,128,device='cuda').bfloat16()
for _ in range(3): A.prompt(q,k,v)
torch.cuda.synchronize()
b=(ctypes.c_longlong*(2*64*8))(); print(gma.lib.gma_clk(b))
import numpy as np
x=np.array(b).reshape(2,64,8)
z=x[0,0,6]
for w in (0,1):
    for n in range(20,26):
        r=x[w,n]; print(w,n,'loop',r[6]-z,'wait',r[0]-r[6],'ld',r[1]-r[0],'max',r[2]-r[1],'resc',r[3]-r[2],'exp',r[4]-r[3],'st',r[5]-r[4])
